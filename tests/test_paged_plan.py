"""The paged attention's shapes (csrc/paged_plan.h), on the CPU: the CTAs that an instantiation is
shaped for fit an SM with all that they need of its shared memory, which is counted here from
the kernel's own arrays, and the cluster form asks for no more CTAs than that."""
import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "row_wise_reduction_gb300", "csrc")
DRIVER = os.path.join(ROOT, "tests", "native", "paged_plan_check.cpp")

SMS, WARPS = 152, 4
SM_SHARED, OPTIN, RESERVED = 228 * 1024, 227 * 1024, 1024  # of an SM; the most of a CTA; the system's of each CTA
WIDTHS = (64, 80, 96, 128, 160, 192, 256)
ROWS = {2: (8, 16), 4: (1, 4, 8)}  # heads of a block, by the element's bytes


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "paged_plan_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, DRIVER, "-o", exe], check=True)

    def run(lines):
        text = "".join(" ".join(str(v) for v in line) + "\n" for line in lines)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(int(v) for v in line.split()) for line in out if line.strip()]

    return run


def need(es, width, rows, stages):
    """A CTA's shared memory with `stages` steps in its rings: dynamic and static."""
    tokens = 16 if es == 2 else 8
    pitch = (width * es // 16 | 1) * 16
    rings = 2 * tokens * pitch * WARPS * stages
    if es == 2:
        joined, scratch = rows * (width + 4) * 4, 0 if width * rows < 2560 else width * rows * 2
    else:
        joined, scratch = rows * width * 4, rows * width * 4 + WARPS * rows * 9 * 4 + 16
    static = 2 * WARPS * rows * 4 + 2 * rows * 4 + WARPS * 2 * 8  # maxima and sums of the warps, of the CTA; found
    return rings + joined + scratch, static


def test_the_ctas_that_shapes_are_made_for_fit_an_sm(plan):
    cases = [(es, width, rows) for es in (2, 4) for width in WIDTHS for rows in ROWS[es]]
    shapes = plan([("s", *c) for c in cases])
    assert len(shapes) == len(cases)
    for (es, width, rows), (tokens, pitch, step, joined, scratch, fixed, ctas, stages) in zip(cases, shapes):
        dynamic, static = need(es, width, rows, stages)
        assert step * stages + rows * joined * 4 + scratch == dynamic
        assert dynamic + static <= OPTIN
        assert ctas * (dynamic + static + RESERVED) <= SM_SHARED, (es, width, rows)
        assert 1 <= ctas <= 3 and 2 <= stages <= 6 and pitch % 32 == 16
        # what gives up a step for company has it; what stands alone could not have had it with two steps
        if ctas == 1:
            dynamic, static = need(es, width, rows, 2)
            assert 2 * (dynamic + static + RESERVED) > SM_SHARED or 2 * step > 104448


def test_clusters_fit_on_the_gpu_at_once(plan):
    asked = list(itertools.product((1, 2, 3, 10, 64), (1, 2, 8, 16, 71), (1, 2, 8), (16, 64, 100, 128, 170, 192, 200, 256),
                                   (1, 500, 5000, 10**6), (0, 300), (2, 4)))
    forms = plan([("f", B, group * kv, kv, D, room, window, es) for B, group, kv, D, room, window, es in asked])
    assert len(forms) == len(asked)
    seen = 0
    for (B, group, kv, D, room, window, es), (cluster, tiles, workspace) in zip(asked, forms):
        rows = (16 if group > 8 else 8) if es == 2 else 8 if group > 4 else 4 if group > 1 else 1
        width = next(w for w in WIDTHS if D <= w)
        units = B * kv * -(-group // rows)
        assert (workspace == 0) == (cluster > 0) and tiles >= 1
        if not cluster:
            continue
        seen += 1
        assert cluster in (1, 2, 4, 8)
        here = plan_ctas(es, width, rows)
        assert units * cluster <= SMS * here, (B, group, kv, D, room, window, es)
    assert seen > 100


def plan_ctas(es, width, rows):
    """CTAs of two steps that share an SM, by their shared memory."""
    dynamic, static = need(es, width, rows, 2)
    return SM_SHARED // (dynamic + static + RESERVED)
