"""Group norm + activation and its backward far from the ordinary values: large
arguments of the activation, means far from zero."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import training as O
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "silu", "gelu", "gelu_tanh"]
FORMS = ["fused", "stream"]
FAR = [0.0, 5.0, 7.25, 7.5, 12.0, 41.0, 43.0, 1e2, 1e4, 1e5, 1e6, 1e7, 1e10, 1e14, 1e18, 1e20]


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, tol, what):
    err = np.abs(got - ref)
    bad = ~(err <= tol)  # a NaN counts
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, at {np.argwhere(bad)[0]} {got[bad][0]} for {ref[bad][0]}"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("through", ["b", "w"])
def test_large_arguments_of_the_activation(act, through, dtype, form, monkeypatch):
    """Channels whose bias, or weight, puts z far out on either side, where value
    and slope are those of a straight line. x lies near +-1, so that no z of
    a large weight comes near 0, where the slope turns within its rounding.
    Bounds as in the operator's other tests: 1e-5 of max(1, |y|), gradients
    2e-5 of the magnitudes that they are added up from, a rounding to bf16
    (2^-8) more."""
    monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    C, G = 2 * len(FAR), len(FAR) // 2
    far = torch.tensor(FAR, dtype=torch.float64)
    for B, S, cut in ((2, 40, C), (1, 33, C - 3)):  # whole vectors; single elements
        g = torch.Generator().manual_seed(6)
        groups = G if cut == C else 1
        sign = torch.where(torch.rand(B, S, cut, generator=g) < 0.5, -1.0, 1.0)
        x = (sign * (1 + 0.1 * torch.rand(B, S, cut, generator=g))).to("cuda", TYPES[dtype])
        dy = torch.randn(B, S, cut, generator=g).to("cuda", TYPES[dtype])
        v = torch.cat([far, -far])[:cut].to("cuda", TYPES[dtype])
        w, b = (v, None) if through == "w" else (None, v)
        if through == "w":  # dz w, and the sums of it over a group, stay within fp32
            w = torch.where(v.abs() > 1e10, torch.ones_like(v), v)
        wn, bn = (None if t is None else f64(t) for t in (w, b))
        stats = torch.empty(B, groups, 2, device="cuda")
        y = ro.rowops_groupnorm_act(x, groups, w, b, act=act, stats=stats)
        u = 2.0**-8 if dtype == "bf16" else 0.0
        ref = O.groupnorm_act(f64(x), groups, wn, bn, name=act)
        near(f64(y), ref, 1e-5 * np.maximum(1, np.abs(ref)) + u * np.abs(ref), "y")
        dx, dw, db = ro.rowops_groupnorm_act_backward(x, dy, stats, groups, w, b, act)
        rdx, rdw, rdb, size, (sw, sb) = O.groupnorm_act_backward(f64(x), f64(dy), groups, wn, bn, name=act)
        near(f64(dx), rdx, 2e-5 * size + u * np.abs(rdx), "dx")
        near(f64(dw), rdw, 2e-5 * sw, "dw")
        near(f64(db), rdb, 2e-5 * sb, "db")


def test_the_activations_keep_a_nan(monkeypatch):
    """A NaN that is not the statistics' own, from w or b, stays in its channel."""
    x = torch.randn(2, 40, 32, device="cuda")
    for form in FORMS:
        monkeypatch.setenv("ROWOPS_GROUPNORM", form)
        for act in ACTS:
            for through in ("w", "b"):
                w, b = torch.ones(32, device="cuda"), torch.zeros(32, device="cuda")
                (w if through == "w" else b)[9] = float("nan")
                stats = torch.empty(2, 4, 2, device="cuda")
                y = ro.rowops_groupnorm_act(x, 4, w, b, act=act, stats=stats)
                assert torch.isnan(y[:, :, 9]).all()
                assert torch.isfinite(y[:, :, 8]).all() and torch.isfinite(y[:, :, 10:]).all()
                dw = ro.rowops_groupnorm_act_backward(x, torch.ones_like(x), stats, 4, w, b, act)[1]
                if act != "none":
                    assert torch.isnan(dw[9]) and torch.isfinite(dw[:8]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,spreads", [("f32", 1e2), ("f32", 1e4), ("f32", 1e6), ("bf16", 1e2)])
@pytest.mark.parametrize("B,S,C,G", [(2, 2048, 64, 4), (1, 40000, 32, 2), (3, 1155, 33, 3), (2, 700, 62, 1)])
def test_group_means_many_spreads_from_zero(B, S, C, G, dtype, spreads, form, monkeypatch):
    """All channels of a group share one mean, `spreads` standard deviations from
    zero: 1 / sd keeps its precision (1e-5, as near zero), the mean is right to 4e-6
    of the spread and its own rounding, and the output is off by that rounding
    (2^-24 |mean|, in spreads) beside the usual 1e-5."""
    monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    rng = np.random.default_rng(8)
    v = rng.normal(size=(B, S, G, C // G)) + spreads * rng.choice([-1.0, 1.0], size=(B, 1, G, 1))
    x = torch.from_numpy(v.reshape(B, S, C)).to("cuda", TYPES[dtype])
    stats = torch.empty(B, G, 2, device="cuda")
    y = ro.rowops_groupnorm_act(x, G, eps=0.0, act="none", stats=stats)
    st, got = O.groupnorm_stats(f64(x), G, 0.0), f64(stats)
    near(got[..., 1] / st[..., 1], np.ones((B, G)), 1e-5, "1 / sd")
    near(got[..., 0], st[..., 0], 4e-6 / st[..., 1] + 2.0**-23 * np.abs(st[..., 0]), "mean")
    ref = O.groupnorm_act(f64(x), G, eps=0.0, name="none")
    wide = np.repeat(2.0**-24 * np.abs(st[..., 0]) * st[..., 1], C // G, axis=1)[:, None]
    u = 2.0**-8 if dtype == "bf16" else 0.0
    near(f64(y), ref, (1e-5 + wide) * np.maximum(1, np.abs(ref)) + u * np.abs(ref), "y")
    z = x.clone()  # in place: the value that the means are kept less of is overwritten in the end
    stats2 = torch.empty_like(stats)
    assert torch.equal(ro.rowops_groupnorm_act(z, G, eps=0.0, act="none", y=z, stats=stats2), y)
    assert torch.equal(stats, stats2)
