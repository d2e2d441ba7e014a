"""GPU parity of group norm + activation and its backward with the 64-bit form.

Tolerances. fp32: the values of a thread's share are added one after another,
at most 64 of them in these shapes, so statistics are off by at most 64 2^-24 =
4e-6 of the spread, and the output, with |act'| <= 1.13 and the activation's
own 1e-6, by 1e-5 |z-scale|, plus what the fp32 mean's own rounding moves x -
mean by (2^-24 |mean| rstd |w|). bf16: a rounding to bf16, 2^-8 relative, more.
Gradients: 2e-5 of the sum of the magnitudes that each is added up from (the
same 4e-6 for the sums, twice, and 1.2e-6 relative for the slope, rounded up),
plus 2^-8 relative for dx in bf16.
"""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import training as O
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "silu", "gelu", "gelu_tanh"]
SENTINEL = 977.0  # no result here equals it


def rows(v, dtype, pad=0, offset=0):
    """The (B, S, C) array on the GPU, positions `pad` elements wider and the
    whole `offset` elements into its storage, all else NaN."""
    B, S, C = v.shape
    ld = C + pad
    base = torch.full((B * S * ld + offset + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    t = torch.as_strided(base, (B, S, C), (S * ld, ld, 1), offset)
    t.copy_(torch.from_numpy(v))
    return t


def f64(t):
    return t.double().cpu().numpy()


def make(B, S, C, G, dtype, pad=0, offset=0, seed=1, mean=0.5):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(B, S, C)) * (0.5 + rng.random(C)) + mean * rng.normal(size=C)
    w = torch.from_numpy(1 + 0.2 * rng.normal(size=C)).to("cuda", TYPES[dtype])
    b = torch.from_numpy(0.1 * rng.normal(size=C)).to("cuda", TYPES[dtype])
    return (rows(x, dtype, pad, offset), rows(rng.normal(size=(B, S, C)), dtype, pad, offset), w, b)


def check(B, S, C, G, dtype, act="silu", pad=0, offset=0, eps=1e-5, affine=True, seed=1, mean=0.5):
    x, dy, w, b = make(B, S, C, G, dtype, pad, offset, seed, mean)
    if not affine:
        w = b = None
    wn, bn = (None, None) if w is None else (f64(w), f64(b))
    xn = f64(x)
    st = O.groupnorm_stats(xn, G, eps)
    per = np.repeat(st[:, None], C // G, axis=2)
    wide = np.abs(1.0 if wn is None else wn)
    floor = 1e-5 + 2.0**-24 * np.abs(per[..., 0]) * per[..., 1] * wide  # the fp32 mean's rounding
    stats = torch.full((B, G, 2), SENTINEL, device="cuda")
    y, buf = out_like(x, offset)
    ro.rowops_groupnorm_act(x, G, w, b, eps, act, y, stats)
    ref = O.groupnorm_act(xn, G, wn, bn, eps, act)
    tol = floor * np.maximum(1, np.abs(ref)) + (2.0**-8 * np.abs(ref) if dtype == "bf16" else 0)
    assert_near(f64(y), ref, tol)
    assert_outside(buf, y)
    # mean to 4e-6 of the spread, 1 / sd to 1e-5
    got = f64(stats)
    assert np.all(np.abs(got[..., 0] - st[..., 0]) <= 4e-6 / st[..., 1] + 2.0**-23 * np.abs(st[..., 0]))
    assert np.all(np.abs(got[..., 1] / st[..., 1] - 1) <= 1e-5)
    # backward
    dx, buf = out_like(x, offset)
    _, dw, db = ro.rowops_groupnorm_act_backward(x, dy, stats, G, w, b, act, dx)
    rdx, rdw, rdb, size, (sw, sb) = O.groupnorm_act_backward(xn, f64(dy), G, wn, bn, eps, act)
    assert_near(f64(dx), rdx, 2e-5 * size + (2.0**-8 * np.abs(rdx) if dtype == "bf16" else 0))
    assert_outside(buf, dx)
    assert_near(f64(dw), rdw, 2e-5 * sw)
    assert_near(f64(db), rdb, 2e-5 * sb)
    return x, dy, w, b, y, stats, dx, dw, db


def out_like(x, offset):
    """An output laid out like x in storage of sentinels."""
    B, S, C = x.shape
    ld = x.stride(1) if S > 1 else max(C, x.stride(0) if B > 1 else C)
    buf = torch.full((B * S * ld + offset + 72,), SENTINEL, dtype=x.dtype, device="cuda")
    return torch.as_strided(buf, (B, S, C), (S * ld, ld, 1), offset), buf


def assert_outside(buf, y):
    mark = torch.zeros(buf.shape, dtype=torch.bool, device="cuda")
    torch.as_strided(mark, y.shape, y.stride(), y.storage_offset()).fill_(True)
    assert torch.all(buf[~mark] == SENTINEL), "written outside its rows"


def assert_near(got, ref, tol):
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"off by {np.max(err / np.maximum(tol, 1e-300)):.3g} of what is allowed"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_activations(dtype, act):
    check(2, 48, 64, 8, dtype, act)
    check(2, 37, 30, 5, dtype, act)  # rows that are no whole vectors


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize(
    "B,S,C,G",
    [(1, 1, 8, 1), (1, 16, 8, 8), (3, 5, 24, 4), (2, 64, 1280, 32), (1, 4096, 320, 32), (2, 1000, 330, 30),
     (1, 9, 8192, 2), (1, 7, 2600, 1), (2, 3, 4104, 27), (5, 17, 1, 1), (4, 100, 3, 3), (300, 4, 16, 2),
     (1, 20000, 32, 4), (70000, 1, 16, 2)])
def test_shapes(dtype, B, S, C, G):
    # (one position of one-channel groups is the next test's)
    check(B, S, C, G, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (8, 8), (5, 3), (40, 0)])
def test_strides_and_alignment(dtype, pad, offset):
    check(2, 50, 96, 6, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", TYPES)
def test_no_affine_and_eps(dtype):
    check(2, 40, 64, 4, dtype, affine=False)
    check(2, 40, 64, 4, dtype, eps=0.0)
    check(2, 40, 64, 4, dtype, eps=3.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_element_path_forced(dtype, monkeypatch):
    monkeypatch.setenv("ROWOPS_KERNEL", "looped")
    check(2, 70, 64, 8, dtype)


def test_groups_of_one_element():
    """Variance 0: xh = 0, so y = act(b) and the gradient of x is exactly 0."""
    x, dy, w, b = make(3, 1, 16, 16, "f32")
    stats = torch.empty(3, 16, 2, device="cuda")
    y = ro.rowops_groupnorm_act(x, 16, w, b, 1e-5, "silu", stats=stats)
    want = O.act(f64(b), "silu")
    assert_near(f64(y), np.broadcast_to(want, y.shape), 1e-6 * np.abs(want) + 1e-7)
    dx, dw, db = ro.rowops_groupnorm_act_backward(x, dy, stats, 16, w, b, "silu")
    assert torch.all(dx == 0) and torch.all(dw == 0)
    assert_near(f64(db), (f64(dy) * O.act_grad(f64(b), "silu")).sum(axis=(0, 1)), 1e-5 * np.abs(f64(dy)).sum((0, 1)))


@pytest.mark.parametrize("mean", [100.0, 3e4])
def test_means_far_from_zero(mean):
    """The variance keeps its precision; the output is off by the fp32 mean's
    rounding at most."""
    check(2, 400, 64, 4, "f32", "none", mean=mean, eps=0.0)


def test_first_value_far_off():
    """A first position of zeros before a map of values near 100."""
    rng = np.random.default_rng(2)
    v = 100 + rng.normal(size=(1, 900, 32))
    v[0, 0] = 0
    x = rows(v, "f32")
    st = O.groupnorm_stats(f64(x), 4, 1e-5)
    stats = torch.empty(1, 4, 2, device="cuda")
    ro.rowops_groupnorm_act(x, 4, act="none", stats=stats)
    assert np.all(np.abs(f64(stats)[..., 1] / st[..., 1] - 1) <= 1e-5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_nan_or_infinity_stays_in_its_group(bad):
    for at in ((0, 0, 9), (0, 30, 9)):
        x, dy, w, b = make(2, 40, 32, 4, "f32")
        clean = ro.rowops_groupnorm_act(x, 4, w, b)
        x[at] = bad
        y = ro.rowops_groupnorm_act(x, 4, w, b)
        assert torch.isnan(y[0, :, 8:16]).all()
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[0, :, 8:16] = False
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place_given_workspace_and_repeatable(dtype):
    x, dy, w, b, y, stats, dx, dw, db = check(3, 500, 320, 32, dtype)
    ws = torch.empty(ro.rowops_groupnorm_act_workspace_bytes(3, 500, 320, 32, x.dtype) + 64, dtype=torch.uint8,
                     device="cuda")
    z = x.clone()
    assert ro.rowops_groupnorm_act(z, 32, w, b, y=z, workspace=ws) is z and torch.equal(z, y)
    again = ro.rowops_groupnorm_act_backward(x, dy, stats, 32, w, b)
    for u, v in zip(again, (dx, dw, db)):
        assert torch.equal(u, v)


def test_gradient_against_differences_of_the_64_bit_form():
    x, dy, w, b = make(1, 20, 24, 3, "f32", seed=7)
    stats = torch.empty(1, 3, 2, device="cuda")
    ro.rowops_groupnorm_act(x, 3, w, b, stats=stats)
    dx = f64(ro.rowops_groupnorm_act_backward(x, dy, stats, 3, w, b)[0])
    xn, h = f64(x), 1e-5
    size = O.groupnorm_act_backward(xn, f64(dy), 3, f64(w), f64(b))[3]
    for at in [(0, 0, 0), (0, 7, 11), (0, 19, 23), (0, 12, 8)]:
        v = xn.copy()
        v[at] += h
        up = (O.groupnorm_act(v, 3, f64(w), f64(b)) * f64(dy)).sum()
        v[at] -= 2 * h
        down = (O.groupnorm_act(v, 3, f64(w), f64(b)) * f64(dy)).sum()
        assert abs((up - down) / (2 * h) - dx[at]) <= 2e-5 * size[at] + 1e-7


def test_empty_batches():
    x = torch.empty(0, 5, 16, device="cuda")
    assert ro.rowops_groupnorm_act(x, 4).shape == (0, 5, 16)
    dx, dw, db = ro.rowops_groupnorm_act_backward(x, x.clone(), torch.empty(0, 4, 2, device="cuda"), 4)
    assert dx.shape == x.shape and torch.all(dw == 0) and torch.all(db == 0)
    x = torch.empty(2, 0, 16, device="cuda")
    assert ro.rowops_groupnorm_act(x, 4).shape == (2, 0, 16)


def test_refusals_of_the_binding():
    x = torch.zeros(2, 6, 16, device="cuda")
    for bad in (x[0], x.transpose(1, 2), x[:, ::2][:, :2], x[:, :4]):
        with pytest.raises(ValueError):
            ro.rowops_groupnorm_act(bad, 4)
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act(x, 4, act="relu")
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act(x, 4, torch.zeros(16, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act(x, 4, stats=torch.zeros(2, 3, 2, device="cuda"))
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act(x, 4, y=torch.empty(2, 6, 32, device="cuda")[..., :16])
    with pytest.raises(TypeError):
        ro.rowops_groupnorm_act(x.half(), 4)
    with pytest.raises(ro.RowopsError):
        ro.rowops_groupnorm_act(x, 5)


def test_one_position():
    """One position has no stride: any that a caller gives does, but its channels must
    be neighbours."""
    x = torch.arange(16, device="cuda").float().view(1, 1, 16)
    want = ro.rowops_groupnorm_act(x, 2)
    far = torch.as_strided(x, (1, 1, 16), (1 << 45, 1 << 45, 1))
    assert torch.equal(ro.rowops_groupnorm_act(far, 2, y=torch.empty_like(x)), want)
    stats = torch.empty(1, 2, 2, device="cuda")
    ro.rowops_groupnorm_act(far, 2, y=torch.empty_like(x), stats=stats)
    dx = ro.rowops_groupnorm_act_backward(far, x, stats, 2, dx=torch.empty_like(x))[0]
    assert torch.equal(dx, ro.rowops_groupnorm_act_backward(x, x, stats, 2)[0])
    spread = torch.zeros(1, 1, 32, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act(x, 2, y=spread)
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act_backward(x, spread, stats, 2)


def test_many_shapes():
    """More shapes than the launch choices that are kept: the same results again."""
    x = torch.randn(1, 700, 32, device="cuda")
    first = [ro.rowops_groupnorm_act(x[:, :s], 4) for s in range(1, 700)]
    for s in (1, 2, 77, 350, 699):
        assert torch.equal(ro.rowops_groupnorm_act(x[:, :s], 4), first[s - 1])


FORMS = ["fused", "stream"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize(
    "B,S,C,G,pad,offset",
    [(2, 64, 1280, 32, 0, 0), (3, 1155, 330, 30, 5, 0), (1, 4096, 320, 32, 0, 0), (9, 1024, 64, 4, 0, 0),
     (2, 5, 96, 12, 0, 0), (1, 3000, 8, 8, 0, 0), (20, 2048, 32, 2, 8, 8), (4, 333, 40, 5, 0, 1), (1, 20000, 16, 1, 0, 0),
     (300, 1, 640, 32, 0, 0), (2, 16, 8192, 8192, 0, 0), (1, 40, 4100, 41, 0, 0)])
def test_both_forms(form, dtype, B, S, C, G, pad, offset, monkeypatch):
    monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    if S == 1 and C == G or (C == G and S < 20):
        # nearly empty groups: the 64-bit variance's own rounding would show
        check(B, S, C, G, dtype, pad=pad, offset=offset, eps=1e-2)
    else:
        check(B, S, C, G, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize(
    "B,S,C,G,pad,offset",
    [(2, 900, 330, 30, 0, 0), (1, 61, 2, 1, 0, 0), (1, 61, 2, 2, 0, 2), (3, 77, 96, 6, 2, 0), (2, 40, 64, 4, 0, 2),
     (1, 13, 4102, 7, 0, 0), (5, 1, 6, 3, 0, 0), (2, 33, 62, 31, 6, 6), (1, 5000, 18, 9, 0, 0)])
def test_two_elements_at_a_time(form, dtype, B, S, C, G, pad, offset, monkeypatch):
    """Even widths, strides and offsets that are no whole vectors'; groups that end
    inside a pair of channels."""
    monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    check(B, S, C, G, dtype, "gelu_tanh", pad=pad, offset=offset, eps=1e-2 if S == 1 else 1e-5)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_both_forms(form, act, monkeypatch):
    monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    for dtype in TYPES:
        check(2, 300, 64, 8, dtype, act)
        check(2, 77, 30, 5, dtype, act)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_samples_streamed(dtype, monkeypatch):
    """Three samples of more than 32 MB: one or a few at a time. Checked against
    the same calls on each sample alone, which the other tests hold to the
    64-bit form, and one sample against that form in sums."""
    monkeypatch.setenv("ROWOPS_GROUPNORM", "stream")
    B, S, C, G = 3, 66000, 256, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, S, C, generator=g, device="cuda").to(TYPES[dtype])
    dy = torch.randn(B, S, C, generator=g, device="cuda").to(TYPES[dtype])
    stats = torch.empty(B, G, 2, device="cuda")
    y = ro.rowops_groupnorm_act(x, G, stats=stats)
    dx, dw, db = ro.rowops_groupnorm_act_backward(x, dy, stats, G)
    v = x.double().reshape(B, S, G, C // G)
    mean = v.mean(dim=(1, 3), keepdim=True)
    xh = (v - mean) / (v.var(dim=(1, 3), keepdim=True, correction=0) + 1e-5).sqrt()
    q = torch.sigmoid(xh)
    u = 2.0**-8 if dtype == "bf16" else 0
    ref = (xh * q).reshape(B, S, C)
    assert torch.all((y - ref).abs() <= 1e-5 * ref.abs().clamp(min=1) + u * ref.abs())
    dz = (dy.double().reshape(v.shape) * (q + xh * q * (1 - q)))
    # a thread adds up to 66000 / 8 positions in turn, but their signs are random: sqrt(8250) 2^-24 of the terms' rms
    # over the square root of their number, far below 2e-5 of the sum of magnitudes
    size = dy.double().abs().reshape(v.shape)
    assert torch.all((db - dz.sum(dim=(0, 1)).reshape(-1)).abs() <= 2e-5 * size.sum(dim=(0, 1)).reshape(-1))
    assert torch.all((dw - (dz * xh).sum(dim=(0, 1)).reshape(-1)).abs()
                     <= 2e-5 * (size * xh.abs()).sum(dim=(0, 1)).reshape(-1))
    rstd = 1 / (v.var(dim=(1, 3), keepdim=True, correction=0) + 1e-5).sqrt()
    rdx = rstd * (dz - dz.mean(dim=(1, 3), keepdim=True) - xh * (dz * xh).mean(dim=(1, 3), keepdim=True))
    rsize = rstd * (size + size.mean(dim=(1, 3), keepdim=True)
                    + xh.abs() * (size * xh.abs()).mean(dim=(1, 3), keepdim=True))
    assert torch.all((dx.reshape(v.shape) - rdx).abs() <= 2e-5 * rsize + u * rdx.abs())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("backward", [False, True])
def test_a_wait_that_runs_out_is_reported(backward, form, monkeypatch):
    """A copy in that never completes, or a sample whose results are never
    announced, ends its wait in a recorded timeout, and the next call is clean."""
    assert ro.rowops_device_status() == 0
    x, dy, w, b = make(2, 512, 64, 4, "bf16")
    stats = torch.empty(2, 4, 2, device="cuda")
    monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    clean = ro.rowops_groupnorm_act(x, 4, w, b, stats=stats)
    cleans = ro.rowops_groupnorm_act_backward(x, dy, stats, 4, w, b)
    assert ro.rowops_device_status() == 0
    monkeypatch.setenv("ROWOPS_WAIT_LIMIT_NS", "20000000")
    monkeypatch.setenv("ROWOPS_TEST_STALL_ROW", "700")
    if backward:
        ro.rowops_groupnorm_act_backward(x, dy, stats, 4, w, b)
    else:
        ro.rowops_groupnorm_act(x, 4, w, b)
    assert ro.rowops_device_status() == 5
    monkeypatch.delenv("ROWOPS_TEST_STALL_ROW")
    assert torch.equal(ro.rowops_groupnorm_act(x, 4, w, b), clean)
    for u, v in zip(ro.rowops_groupnorm_act_backward(x, dy, stats, 4, w, b), cleans):
        assert torch.equal(u, v)
    assert ro.rowops_device_status() == 0
