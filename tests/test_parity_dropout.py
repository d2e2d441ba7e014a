"""GPU parity of bias + dropout + residual and its backward with the 64-bit
form, whose generator is pinned by the published answers. The mask is compared
exactly. Values: (x + b), its product with the scale and the sum with the
residual round once each, so fp32 is off by at most 3 2^-24 (|x| + |b|) s +
|r|) and bf16 by one rounding, 2^-8, more. dbias: at most 2^14 terms in any one
order, of which a thread adds at most 600 in turn: 600 2^-24 = 4e-5 of the sum of
magnitudes."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import training as O
from tests import _compare as C
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def place(M, N, dtype, pad, offset, seed):
    g = torch.Generator().manual_seed(seed)
    base = torch.full((M * (N + pad) + offset + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    t = torch.as_strided(base, (M, N), (N + pad, 1), offset)
    t.copy_(torch.randn(M, N, generator=g))
    return t


def near(got, ref, size, dtype, rel=3 * 2.0**-24):
    tol = rel * size + (2.0**-8 * np.abs(ref) if dtype == "bf16" else 0)
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"off by {np.max(err / np.maximum(tol, 1e-300)):.3g} of what is allowed"


def check(M, N, dtype, p=0.1, bias=True, residual=True, pad=0, offset=0, seed=11, off=3):
    x = place(M, N, dtype, pad, offset, 1)
    r = place(M, N, dtype, pad, offset, 2) if residual else None
    b = torch.randn(N, generator=torch.Generator().manual_seed(3)).to("cuda", TYPES[dtype]) if bias else None
    keep = O.dropout_keep(np.arange(M), N, p, seed, off)
    scale = O.dropout_scale(p)
    xn, rn, bn = (None if t is None else C.to_f64(t) for t in (x, r, b))
    y, buf, inside = gu.guarded_like(x, offset=offset)
    ro.rowops_bias_dropout_residual(x, r, b, p, seed, off, y)
    ref = O.bias_dropout_residual(xn, rn, bn, keep, p)
    size = keep * (np.abs(xn) + (0 if bn is None else np.abs(bn))) * scale + (0 if rn is None else np.abs(rn))
    near(C.to_f64(y), ref, size, dtype)
    gu.assert_guard_untouched(buf, inside)
    if rn is not None:  # what is dropped leaves the residual as it is
        assert np.array_equal(C.to_f64(y)[~keep], rn[~keep])
    else:
        assert np.all(C.to_f64(y)[~keep] == 0)
    dx, buf, inside = gu.guarded_like(x, offset=offset)
    _, db = ro.rowops_bias_dropout_residual_backward(x, p, seed, off, dx, bias_grad=bias)
    rdx = np.where(keep, xn * scale, 0)
    near(C.to_f64(dx), rdx, np.abs(rdx), dtype)
    gu.assert_guard_untouched(buf, inside)
    if bias:
        assert np.all(np.abs(C.to_f64(db) - rdx.sum(axis=0)) <= 4e-5 * np.abs(rdx).sum(axis=0))
    return x, r, b, y, dx, db


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 3, 7, 8, 9, 16, 31, 40, 64, 100, 127, 256, 330, 768, 1000, 4097, 8192])
def test_widths(dtype, N):
    check(37, N, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (1, 8192), (2, 20000), (70001, 8), (5000, 33), (16385, 256), (3, 100000)])
def test_heights(dtype, M, N):
    check(M, N, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [0.0, 1e-6, 1e-5, 0.25, 0.5, 0.9999, 1.0])
def test_probabilities(dtype, p):
    check(50, 264, dtype, p)
    check(50, 77, dtype, p)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (False, False)])
def test_optional_inputs(dtype, bias, residual):
    check(40, 512, dtype, bias=bias, residual=residual)
    check(40, 45, dtype, bias=bias, residual=residual)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (5, 0), (0, 1), (8, 8), (3, 3), (0, 4)])
def test_strides_and_alignment(dtype, pad, offset):
    check(41, 320, dtype, pad=pad, offset=offset)
    check(41, 50, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("seed,off", [(0, 0), (-1, 1), ((1 << 64) - 1, (1 << 64) - 1), (1 << 40, 1 << 33)])
def test_wide_seeds_and_offsets(seed, off):
    check(16, 64, "f32", 0.5, seed=seed, off=off)


def test_the_mask_is_the_same_for_every_layout_and_type():
    masks = []
    for dtype in TYPES:
        for pad, offset in ((0, 0), (3, 1), (8, 0)):
            x = place(65, 200, dtype, pad, offset, 4)
            x.fill_(1)
            masks.append((ro.rowops_bias_dropout_residual(x, p=0.3, seed=8, offset=9) != 0).cpu())
            masks.append((ro.rowops_bias_dropout_residual(x[:, :130], p=0.3, seed=8, offset=9) != 0).cpu())
    for m in masks:
        assert torch.equal(m, masks[0][:, : m.shape[1]])


@pytest.mark.parametrize("dtype", TYPES)
def test_dropped_places_may_hold_anything(dtype):
    x = place(64, 96, dtype, 0, 0, 5)
    keep = torch.from_numpy(O.dropout_keep(np.arange(64), 96, 0.5, 1, 2)).cuda()
    r = torch.ones_like(x)
    for bad in (float("nan"), float("inf")):
        z = torch.where(keep, x, torch.full_like(x, bad))
        y = ro.rowops_bias_dropout_residual(z, r, p=0.5, seed=1, offset=2)
        assert torch.isfinite(y).all() and torch.all(y[~keep] == 1)
        dx, db = ro.rowops_bias_dropout_residual_backward(z, 0.5, 1, 2)
        assert torch.isfinite(dx.float()).all() and torch.isfinite(db).all()
    z = torch.full_like(x, float("nan"))
    assert torch.all(ro.rowops_bias_dropout_residual(z, r, p=1.0) == 1)


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place_and_repeatable(dtype):
    x, r, b, y, dx, db = check(300, 1032, dtype)
    z = x.clone()
    assert torch.equal(ro.rowops_bias_dropout_residual(z, r, b, 0.1, 11, 3, z), y)
    z = r.clone()
    assert torch.equal(ro.rowops_bias_dropout_residual(x, z, b, 0.1, 11, 3, z), y)
    z = x.clone()
    dz, dc = ro.rowops_bias_dropout_residual_backward(z, 0.1, 11, 3, z)
    assert torch.equal(dz, dx) and torch.equal(dc, db)


def test_device_offset_in_a_replayed_graph():
    x = torch.ones(128, 256, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    db = torch.empty(256, device="cuda")
    ws = torch.empty(ro.rowops_bias_dropout_residual_backward_workspace_bytes(128, 256, x.dtype), dtype=torch.uint8,
                     device="cuda")
    at = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        ro.rowops_bias_dropout_residual(x, None, None, 0.5, 3, 10, y, device_offset=at)
        ro.rowops_bias_dropout_residual_backward(x, 0.5, 3, 10, dx, db, device_offset=at, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in (0, 1, -3, 1 << 40):
        at.fill_(k)
        g.replay()
        want = O.dropout_keep(np.arange(128), 256, 0.5, 3, 10 + k)
        assert np.array_equal((y != 0).cpu().numpy(), want) and torch.equal(y, dx)
        assert np.array_equal(db.cpu().numpy(), 2.0 * want.sum(axis=0))


def test_no_rows_and_refusals():
    x = torch.empty(0, 24, device="cuda")
    assert ro.rowops_bias_dropout_residual(x).shape == (0, 24)
    dx, db = ro.rowops_bias_dropout_residual_backward(x)
    assert dx.shape == (0, 24) and torch.all(db == 0)
    x = torch.zeros(4, 24, device="cuda")
    with pytest.raises(ro.RowopsError):
        ro.rowops_bias_dropout_residual(x, p=1.5)
    with pytest.raises(ValueError):
        ro.rowops_bias_dropout_residual(x, torch.zeros(4, 25, device="cuda"))
    with pytest.raises(ValueError):
        ro.rowops_bias_dropout_residual(x, bias=torch.zeros(23, device="cuda"))
    with pytest.raises(ValueError):
        ro.rowops_bias_dropout_residual(x, device_offset=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        ro.rowops_bias_dropout_residual_backward(x, dbias=torch.zeros(24, device="cuda"), bias_grad=False)


@pytest.mark.parametrize("what", ["y", "residual", "dx"])
def test_one_row_of_spread_columns_is_refused(what):
    """A single row has no row stride to compare, but its columns must be neighbours."""
    x = torch.ones(1, 24, device="cuda")
    spread = torch.zeros(1, 48, device="cuda")[:, ::2]
    with pytest.raises(ValueError):
        if what == "y":
            ro.rowops_bias_dropout_residual(x, y=spread)
        elif what == "residual":
            ro.rowops_bias_dropout_residual(x, spread)
        else:
            ro.rowops_bias_dropout_residual_backward(x, dx=spread)
    wide = torch.as_strided(torch.zeros(24, device="cuda"), (1, 24), (1000, 1))  # its stride leads nowhere: no matter
    assert torch.equal(ro.rowops_bias_dropout_residual(x, wide, p=0.0, y=torch.empty_like(wide)), x)
