"""Calls of the serving operators that their documentation allows and that are easily forgotten: caches whose heads
are one head expanded, or that are one tensor, pages shared by sequences and met twice in one, weights off 16 bytes,
a residual that is the input itself, dimensions of one entry with any stride, equal calls."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import serving as O
from tests import _compare as C
from tests import gpu_util as gu
from tests.test_parity_paged_attention import LINE, TYPES, hold as hold_attention, problem
from tests.test_parity_rmsnorm_quant import hold as hold_norm, place

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


def attend(q, k, v, table, n, **more):
    lse = torch.empty(q.shape[:2], device="cuda")
    out = ro.rowops_paged_attention(q, k, v, table, n, lse=lse, **more)
    hold_attention(out, lse, q, k, v, table, n, more.get("scale"), more.get("window", 0))
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [9, LINE])
def test_heads_expanded_and_one_cache_for_both(dtype, width):
    q, k, v, table, n = problem([130, 0, 77], 8, 1, 64, 16, dtype, width=width)
    one = attend(q, k, v, table, n)
    many = attend(q, k.expand(-1, -1, 4, -1), v.expand(-1, -1, 4, -1), table, n)  # two heads to each of four
    assert torch.allclose(one.float(), many.float(), rtol=2.0**-7, atol=1e-5)
    attend(q, k, k, table, n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [30, LINE])
def test_pages_shared_and_met_twice(dtype, width):
    q, k, v, table, n = problem([300, 290, 17], 8, 2, 80, 16, dtype, width=width)
    table[1, :10] = table[0, :10]
    table[0, 12] = table[0, 3]
    table[2, 1] = table[2, 0]
    v[table[2, 1].long(), 1:] = 1.0  # (slots that only the second meeting reaches)
    k[table[2, 1].long(), 1:] = 0.5
    attend(q, k, v, table, n)
    attend(q, k, v, table, n, window=100)


@pytest.mark.parametrize("dtype", TYPES)
def test_dimensions_of_one_entry_have_any_stride(dtype):
    q, k, v, table, n = problem([60], 3, 1, 40, 64, dtype)
    want = attend(q, k, v, table, n)
    strange = lambda t, *at: t.as_strided(t.shape, tuple(999983 if i in at else s for i, s in enumerate(t.stride())))
    assert k.shape[2] == 1 and table.shape[1] == 1
    assert torch.equal(want, attend(strange(q, 0), strange(k, 2), strange(v, 2), strange(table, 0, 1), n))
    pool = int(table[0, 0])
    assert torch.equal(want, attend(q, strange(k[pool:pool + 1], 0, 2), strange(v[pool:pool + 1], 0, 2), torch.zeros_like(table), n))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1024, 1026, 1031, 40000])
@pytest.mark.parametrize("group", [0, 64, 96])
def test_weights_off_16_bytes_and_the_input_as_residual(dtype, N, group):
    g = torch.Generator().manual_seed(N)
    x = place(torch.randn(50, N, generator=g), dtype)
    for offset in (0, 1, 2, 8):
        w = torch.randn(N + 8, generator=g).to("cuda", TYPES[dtype])[offset:offset + N]
        q, scales, s = ro.rowops_rmsnorm_quant(x, x, w, 1e-5, group)
        assert torch.equal(s, (x.float() + x.float()).to(x.dtype))
        hold_norm(q, scales, C.to_f64(s), C.to_f64(w), group)
        y = x.clone()
        q2, scales2, s2 = ro.rowops_rmsnorm_quant(y, y, w, 1e-5, group, residual_out=y)
        assert torch.equal(s2, s) and torch.equal(scales2, scales) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES)
def test_numbers_and_tensors_mixed_among_the_knobs(dtype):
    g = torch.Generator().manual_seed(3)
    x = place(2 * torch.randn(20, 3000, generator=g), dtype)
    u = torch.rand(20, generator=g).cuda()
    full = lambda v, t=torch.float32: torch.full((20,), v, dtype=t, device="cuda")
    want = ro.rowops_sample(x, u, temperature=0.75, top_k=50, top_p=0.875, min_p=0.03125)
    for mask in range(16):
        knobs = dict(temperature=full(0.75) if mask & 1 else 0.75, top_k=full(50, torch.int32) if mask & 2 else 50,
                     top_p=full(0.875) if mask & 4 else 0.875, min_p=full(0.03125) if mask & 8 else 0.03125)
        assert torch.equal(want, ro.rowops_sample(x, u, **knobs))
    # one tensor for several of them, u among them
    same = full(0.5)
    assert torch.equal(ro.rowops_sample(x, same, temperature=same, top_p=same, min_p=same),
                       ro.rowops_sample(x, full(0.5), temperature=0.5, top_p=0.5, min_p=0.5))
    for i in range(20):
        token, _, margin = O.sample_row(C.to_f64(x[i]), float(u[i]), 0.75, 50, 0.875, 0.03125)
        assert int(want[i]) == token or margin < 2.0**-28


def test_equal_calls_give_equal_bits():
    q, k, v, table, n = problem([900, 1, 333] + [50] * 100, 16, 2, 128, 16, "bf16")
    x, u = torch.randn(64, 50000, device="cuda"), torch.rand(64, device="cuda")
    first = None
    for _ in range(20):
        lse, lp = torch.empty(103, 16, device="cuda"), torch.empty(64, device="cuda")
        got = [ro.rowops_paged_attention(q, k, v, table, n, lse=lse), lse, ro.rowops_sample(x, u, top_k=99, top_p=0.8, logprob=lp), lp]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    assert np.isfinite(first[1].cpu().numpy()).all()
