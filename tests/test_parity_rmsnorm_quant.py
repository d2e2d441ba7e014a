"""GPU parity of RMSNorm with an 8-bit result with its 64-bit form. residual_out is
the fp32 sum rounded once, compared exactly. The sum of squares is added up in chains of
at most max(64, N / 512) + 32 terms in fp32, of whose error the root takes half; the
root, the products and the quotient add at most 8 roundings: a relative error of
(chain / 2 + 8) 2^-24 in y, the scales and y / scale. Rounding to e4m3 then moves
y / scale by half a step at most."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import serving as O
from tests import _compare as C
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def place(v, dtype, pad=0, offset=0):
    M, N = v.shape
    base = torch.full((M * (N + pad) + offset + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    t = torch.as_strided(base, (M, N), (N + pad, 1), offset)
    t.copy_(v)
    return t


def normal(M, N, seed):
    return torch.randn(M, N, generator=torch.Generator().manual_seed(seed))


def relative(N):
    return ((max(64, N / 512) + 32) / 2 + 8) * 2.0**-24


def hold(q, scales, s, w, group, eps=1e-5):
    """q and scales for the summed rows s (as stored)."""
    M, N = s.shape
    y = O.rmsnorm(s, w, eps)
    want = O.quant_scales(y, group)
    got = scales.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= relative(N) * want + 2.0**-149)
    v = y / np.repeat(want, group or N, axis=1)[:, :N]
    n = q.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(n - v) <= O.e4m3_half_step(v) + 2 * relative(N) * np.abs(v))


def check(M, N, dtype, group=0, residual=True, weight=True, pad=0, offset=0, qpad=0, qoffset=0):
    x, r = place(normal(M, N, 1), dtype, pad, offset), place(3 * normal(M, N, 2), dtype, pad, offset)
    w = (1 + 0.2 * normal(1, N, 3)[0]).to("cuda", TYPES[dtype]) if weight else None
    base = torch.full((M * (N + qpad) + qoffset + 32,), 0x55, dtype=torch.uint8, device="cuda")
    q = torch.as_strided(base.view(torch.float8_e4m3fn), (M, N), (N + qpad, 1), qoffset + 16)
    out, buf, inside = gu.guarded_like(x, offset=offset)
    q2, scales, s = ro.rowops_rmsnorm_quant(x, r if residual else None, w, 1e-5, group, q,
                                            residual_out=out if residual else None)
    assert q2 is q and scales.shape == (M, -(-N // group) if group else 1)
    if residual:
        assert s is out and torch.equal(s, (x.float() + r.float()).to(x.dtype))
        gu.assert_guard_untouched(buf, inside)
    else:
        assert s is None
    hold(q, scales, C.to_f64(s if residual else x), None if w is None else C.to_f64(w), group)
    mark = torch.full_like(base, 0)
    torch.as_strided(mark, (M, N), (N + qpad, 1), qoffset + 16).fill_(1)
    assert torch.all(base[mark == 0] == 0x55), "a kernel wrote outside q's rows"
    return x, r, w, q, scales, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("N", [1, 7, 31, 32, 33, 64, 127, 128, 256, 1000, 4099, 8192])
def test_widths(dtype, group, N):
    check(19, N, dtype, group)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("N", [16384, 20000, 40000, 100003])
def test_long_rows(dtype, group, N):
    check(3, N, dtype, group)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(1, 4096), (1, 1), (2, 8192), (5000, 64), (3001, 256), (300, 5120), (70001, 32)])
def test_heights(dtype, M, N):
    check(M, N, dtype, 0)
    check(M, N, dtype, 32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [96, 160, 192, 256, 512, 1024, 4096, 1 << 20])
def test_groups(dtype, group):
    check(9, 2048, dtype, group) if group <= 2048 else check_whole(dtype, group)


def check_whole(dtype, group):
    """Groups of the row's length and more are the row."""
    x = place(normal(9, 2048, 1), dtype)
    q, scales, _ = ro.rowops_rmsnorm_quant(x, group=group)
    q0, scales0, _ = ro.rowops_rmsnorm_quant(x)
    assert torch.equal(scales, scales0) and torch.equal(q.view(torch.uint8), q0.view(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual,weight", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("N,group", [(512, 0), (512, 64), (300, 0), (301, 32)])
def test_optional_inputs(dtype, residual, weight, N, group):
    check(40, N, dtype, group, residual, weight)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset,qpad,qoffset", [(8, 0, 0, 0), (5, 0, 0, 0), (0, 1, 0, 0), (8, 8, 16, 0), (3, 3, 1, 1),
                                                     (0, 0, 4, 2), (0, 4, 8, 8)])
def test_strides_and_alignment(dtype, pad, offset, qpad, qoffset):
    for N, group in ((320, 0), (320, 64), (50, 32)):
        check(23, N, dtype, group, True, True, pad, offset, qpad, qoffset)
        check(23, N, dtype, group, False, True, pad, offset, qpad, qoffset)


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place_and_repeatable(dtype):
    for N, group in ((1024, 128), (1031, 0)):
        x, r, w, q, scales, s = check(33, N, dtype, group)
        for target in ("x", "residual"):
            a, b = x.clone(), r.clone()
            q2, scales2, s2 = ro.rowops_rmsnorm_quant(a, b, w, 1e-5, group, residual_out=a if target == "x" else b)
            assert torch.equal(q2.view(torch.uint8), q.contiguous().view(torch.uint8))
            assert torch.equal(scales2, scales) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [256, 259, 40000])
def test_nothing_and_not_a_number(dtype, N):
    x = place(normal(6, N, 5), dtype)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, N - 1] = float("inf")
    x[4] *= 1e-30
    x[5, : min(N, 64)] = 0
    for group in (0, 64):
        q, scales, _ = ro.rowops_rmsnorm_quant(x, group=group)
        n = q.float()
        assert torch.all(n[1] == 0) and torch.all(scales[1] == 2.0**-126)
        assert torch.isnan(n[2]).all() and torch.isnan(scales[2]).all()
        # an infinity: the root is infinite, so what is finite becomes s / inf = 0, and inf / inf NaN
        last = (N - 1) // group * group if group else 0
        assert torch.isnan(n[3, last:]).all() and torch.isnan(scales[3, -1])
        assert torch.all(n[3, :last] == 0) and torch.all(scales[3, :-1] == 2.0**-126)
        rows = [0, 4, 5]
        hold(q[rows], scales[rows], C.to_f64(x[rows]), None, group)


def test_a_long_tail_of_small_numbers_keeps_its_own_scale():
    """An outlier costs its own group alone its precision."""
    x = place(normal(4, 512, 6), "f32")
    x[:, 5] = 1e4
    q, scales, _ = ro.rowops_rmsnorm_quant(x, group=128)
    hold(q, scales, C.to_f64(x), None, 128)
    y = O.rmsnorm(C.to_f64(x), None, 1e-5)
    back = q.double().cpu().numpy() * np.repeat(scales.double().cpu().numpy(), 128, axis=1)
    assert np.all(np.abs(back - y)[:, 128:] <= 2.0**-4 * 1.001 * np.abs(y[:, 128:]) + scales.max().item() * 2.0**-10)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    for call in (lambda: ro.rowops_rmsnorm_quant(x, group=48), lambda: ro.rowops_rmsnorm_quant(x, eps=-1.0)):
        with pytest.raises(ro.RowopsError):
            call()
    for call in (lambda: ro.rowops_rmsnorm_quant(x, torch.zeros(4, 65, device="cuda")),
                 lambda: ro.rowops_rmsnorm_quant(x, w=torch.zeros(63, device="cuda")),
                 lambda: ro.rowops_rmsnorm_quant(x, residual_out=torch.zeros_like(x)),
                 lambda: ro.rowops_rmsnorm_quant(x, q=torch.zeros(4, 64, dtype=torch.uint8, device="cuda")),
                 lambda: ro.rowops_rmsnorm_quant(x, scales=torch.zeros(5, device="cuda")),
                 lambda: ro.rowops_rmsnorm_quant(x.cpu()),
                 lambda: ro.rowops_rmsnorm_quant(x[:, ::2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ro.rowops_rmsnorm_quant(x.half())
    q, scales, s = ro.rowops_rmsnorm_quant(x[:0], x[:0], group=32)
    assert q.shape == (0, 64) and scales.shape == (0, 2) and s.shape == (0, 64)
