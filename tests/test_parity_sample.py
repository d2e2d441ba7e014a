"""GPU parity of sampling with its 64-bit form: the same tokens, wherever no decision of
the row could be turned by a relative error of 2^-28 in the weights (they are right to
2^-29 of their value and 2^-45 of the largest). logprob within 2^-22 of
its magnitude and 2^-28 for the sum."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import serving as O
from tests import _compare as C
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KNOBS = ("temperature", "top_k", "top_p", "min_p")


def place(v, dtype, pad=0, offset=0):
    M, N = v.shape
    base = torch.full((M * (N + pad) + offset + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    t = torch.as_strided(base, (M, N), (N + pad, 1), offset)
    t.copy_(v)
    return t


def rows(M, N, seed, spread=2.5):
    return spread * torch.randn(M, N, generator=torch.Generator().manual_seed(seed))


def uniform(M, seed):
    return torch.rand(M, generator=torch.Generator().manual_seed(seed)).cuda()


def check(x, u, **knobs):
    """Equal tokens and log-probabilities; returns the tokens."""
    M, N = x.shape
    logprob = torch.full((M + 2,), 7.0, device="cuda")
    token = torch.full((M + 2,), -9, dtype=torch.int64, device="cuda")
    ro.rowops_sample(x, u, **knobs, token=token[1:-1], logprob=logprob[1:-1])
    assert token[0] == -9 and token[-1] == -9 and logprob[0] == 7 and logprob[-1] == 7
    xs, us = C.to_f64(x), u.double().cpu().numpy()
    each = {k: (v.double().cpu().numpy() if isinstance(v, torch.Tensor) else np.full(M, np.float64(np.float32(v))))
            for k, v in knobs.items()}
    near = 0
    for i in range(M):
        want, lp, margin = O.sample_row(xs[i], us[i], **{k: (int(v[i]) if k == "top_k" else v[i]) for k, v in each.items()})
        if margin < 2.0**-28:
            near += 1
            continue
        got, glp = int(token[i + 1]), float(logprob[i + 1])
        assert got == want, f"row {i}: {got}, not {want} (margin {margin:.2g})"
        assert np.isnan(lp) == np.isnan(glp) and (np.isnan(lp) or abs(glp - lp) <= 2.0**-22 * abs(lp) + 2.0**-28)
    assert near <= M // 50
    return token[1:-1].clone()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 2, 7, 31, 32, 33, 100, 255, 1000, 4097, 32000, 50021])
def test_widths(dtype, N):
    x, u = place(rows(24, N, 1), dtype), uniform(24, 2)
    check(x, u)
    check(x, u, temperature=0.7, top_k=min(N, 20))
    check(x, u, temperature=1.3, top_p=0.8)
    check(x, u, min_p=0.05)
    check(x, u, temperature=0.8, top_k=40, top_p=0.9, min_p=0.02)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [65536, 131072, 200000, 327680])
def test_long_rows(dtype, N):
    x, u = place(rows(5, N, 3), dtype), uniform(5, 4)
    check(x, u)
    check(x, u, temperature=0.6, top_p=0.95)
    check(x, u, top_k=5000, top_p=0.5, min_p=1e-4)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows(dtype):
    x, u = place(rows(3000, 257, 5), dtype), uniform(3000, 6)
    check(x, u, top_k=30, top_p=0.7)
    x, u = place(rows(1, 8192, 5), dtype), uniform(1, 6)
    check(x, u, top_k=30, top_p=0.7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [2000, 70001])
def test_knobs_by_row(dtype, N):
    M = 64 if N < 10000 else 24
    g = torch.Generator().manual_seed(7)
    x, u = place(rows(M, N, 8), dtype), uniform(M, 9)

    def half(v):
        return torch.where(torch.rand(M, generator=g) < 0.5, v, torch.zeros_like(v)).cuda()

    temperature = half(0.3 + torch.rand(M, generator=g))
    top_k = half(torch.randint(1, 300, (M,), generator=g, dtype=torch.int32))
    top_p = 1 - half(torch.rand(M, generator=g))
    min_p = half(0.3 * torch.rand(M, generator=g))
    check(x, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    check(x, u, temperature=temperature, top_p=top_p)
    check(x, u, top_k=top_k, temperature=0.9)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [1, 2, 3, 50, 999, 1000, 1001, 1 << 30])
def test_top_k(dtype, k):
    x, u = place(rows(40, 1000, 10), dtype), uniform(40, 11)
    check(x, u, top_k=k)
    check(x, u, top_k=k, temperature=50.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [0.0, 1e-9, 0.01, 0.5, 0.999, 0.9999999, 1.0, 2.0])
def test_top_p(dtype, p):
    x, u = place(rows(40, 3000, 12), dtype), uniform(40, 13)
    check(x, u, top_p=p)
    check(x, u, top_p=p, top_k=100)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [0.0, 1e-30, 1e-4, 0.3, 0.999, 1.0])
def test_min_p(dtype, p):
    x, u = place(rows(40, 3000, 14), dtype), uniform(40, 15)
    check(x, u, min_p=p)
    check(x - 30, u, min_p=p, temperature=0.4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("temperature", [0.0, 1e-20, 1e-3, 0.1, 1.0, 10.0, 1e4, 1e30, float("inf")])
def test_temperatures(dtype, temperature):
    x, u = place(rows(40, 1500, 16), dtype), uniform(40, 17)
    check(x, u, temperature=temperature)
    if temperature > 0:
        check(x, u, temperature=temperature, top_k=77)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (8, 8)])
def test_strides_and_alignment(dtype, pad, offset):
    u = uniform(16, 18)
    for N in (640, 777, 40001):
        plain = check(place(rows(16, N, 19), dtype), u, top_k=50, top_p=0.9)
        assert torch.equal(plain, check(place(rows(16, N, 19), dtype, pad, offset), u, top_k=50, top_p=0.9))


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_logits(dtype):
    """Ties go by index, and borders are exact: n equal columns share [0, 1) evenly."""
    for n in (1, 2, 4, 256):
        x = torch.full((n, 1000), -3.0)
        x[:, 100:100 + 3 * n:3] = 2.0  # n of them far above the rest
        x = place(x, dtype)
        u = (torch.arange(n, dtype=torch.float32) / n).cuda()
        want = 100 + 3 * torch.arange(n, device="cuda")
        assert torch.equal(ro.rowops_sample(x, u, top_k=n), want)
        assert torch.equal(ro.rowops_sample(x, u, min_p=0.5), want)
        below = torch.nextafter(u + 1.0 / n, torch.zeros(1, device="cuda"))
        assert torch.equal(ro.rowops_sample(x, below, top_k=n), want)
        if n >= 4:  # half of them: the first ones
            assert torch.equal(ro.rowops_sample(x, u, top_k=n // 2), (100 + 3 * (torch.arange(n, device="cuda") // 2)))
            assert torch.equal(ro.rowops_sample(x, u, top_k=n, top_p=0.5), (100 + 3 * (torch.arange(n, device="cuda") // 2)))
    x = place(torch.zeros(8, 60000), dtype)
    x[:, 1::2] = -0.0  # equal to 0
    u = (torch.arange(8, dtype=torch.float32) / 8).cuda()
    assert torch.equal(ro.rowops_sample(x, u), 7500 * torch.arange(8, device="cuda"))
    assert torch.equal(ro.rowops_sample(x, u, top_k=16), 2 * torch.arange(8, device="cuda"))
    assert torch.equal(ro.rowops_sample(x, u, temperature=0), torch.zeros(8, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [300, 70000])
def test_masks_infinities_and_not_a_number(dtype, N):
    low = torch.finfo(TYPES[dtype]).min
    x = rows(10, N, 20)
    x[0, :] = -float("inf")
    x[1, 17] = float("nan")
    x[2, :-1] = -float("inf")        # one column left
    x[3, 5:] = low                   # masked by the type's lowest value
    x[4, :] = low                    # all of them: evenly
    x[5, [9, 40, 200]] = float("inf")  # alone, evenly
    x[6, : N // 2] = -float("inf")
    x[7, :] = -float("inf")
    x[7, [3, N - 1]] = 1.5
    x[8, N - 1] = float("nan")
    x = place(x, dtype)
    u = uniform(10, 21)
    for knobs in ({}, dict(top_k=8), dict(top_p=0.9), dict(min_p=0.1), dict(top_k=N - 1, top_p=0.99, min_p=0.001)):
        t = check(x, u, **knobs)
        assert t[0] == -1 and t[1] == -1 and t[8] == -1 and t[2] == N - 1
        assert int(t[5]) in (9, 40, 200) and int(t[7]) in (3, N - 1) and int(t[3]) < 5
    t = ro.rowops_sample(x, u, temperature=0)
    assert t[0] == -1 and t[1] == -1 and t[8] == -1 and t[2] == N - 1 and t[5] == 9 and t[7] == 3 and t[4] == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_numbers_outside_their_ranges(dtype):
    x = place(rows(6, 500, 22), dtype)
    nan, inf = float("nan"), float("inf")
    lo, hi = torch.zeros(6, device="cuda"), torch.full((6,), 1 - 2.0**-24, device="cuda")
    for u, like in (([-1.0, -0.0, nan, -inf, -1e-30, 0.0], lo), ([1.0, 2.0, inf, 1e30, 1.0, 5.0], hi)):
        got = ro.rowops_sample(x, torch.tensor(u, device="cuda"), top_k=20)
        assert torch.equal(got, ro.rowops_sample(x, like, top_k=20))
    u = uniform(6, 23)
    t = torch.tensor([-1.0, nan, -inf, 0.0, -0.0, -5.0], device="cuda")
    assert torch.equal(ro.rowops_sample(x, u, temperature=t), ro.rowops_sample(x, u, temperature=0.0))
    k = torch.tensor([-3, 0, 500, 501, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    assert torch.equal(ro.rowops_sample(x, u, top_k=k), ro.rowops_sample(x, u))
    p = torch.tensor([1.0, 1.5, inf, nan, 7.0, 1.0], device="cuda")
    assert torch.equal(ro.rowops_sample(x, u, top_p=p), ro.rowops_sample(x, u))
    p = torch.tensor([0.0, -1.0, -inf, -0.0, -1e-9, 0.0], device="cuda")
    assert torch.equal(ro.rowops_sample(x, u, top_p=p), ro.rowops_sample(x, u, temperature=0))
    p = torch.tensor([0.0, -1.0, nan, -inf, -0.0, -2.0], device="cuda")
    assert torch.equal(ro.rowops_sample(x, u, min_p=p), ro.rowops_sample(x, u))
    p = torch.tensor([1.0, 1.5, inf, 2.0, 1.0, 3.0], device="cuda")
    assert torch.equal(ro.rowops_sample(x, u, min_p=p), ro.rowops_sample(x, u, temperature=0))


@pytest.mark.parametrize("dtype", TYPES)
def test_frequencies(dtype):
    """Evenly spaced numbers u draw each token as often as its probability says, to one draw."""
    x = rows(1, 200, 24)
    M = 4096
    u = ((torch.arange(M, dtype=torch.float32) + 0.5) / M).cuda()
    t = ro.rowops_sample(place(x.expand(M, -1), dtype), u, temperature=0.9)
    p = torch.softmax(x[0].to(TYPES[dtype]).double() / float(np.float32(0.9)), dim=0)
    got = torch.bincount(t.cpu(), minlength=200).double() / M
    assert torch.all((got - p).abs() <= 1.0 / M + 1e-7)
    assert torch.equal(t.sort().values, t)


def test_the_same_alone_on_a_stream_and_in_a_replayed_graph():
    x, u = place(rows(9, 40000, 25), "bf16"), uniform(9, 26)
    knobs = dict(temperature=0.8, top_k=100, top_p=0.9)
    t = check(x, u, **knobs)
    for i in (0, 4, 8):
        assert torch.equal(ro.rowops_sample(x[i:i + 1], u[i:i + 1], **knobs), t[i:i + 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = ro.rowops_sample(x, u, **knobs, stream=s)
    s.synchronize()
    assert torch.equal(again, t)
    token = torch.empty_like(t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ro.rowops_sample(x, u, **knobs, token=token)
    for seed in (30, 31):
        u.copy_(uniform(9, seed))
        g.replay()
        assert torch.equal(token, check(x, u, **knobs))


def test_refusals():
    x, u = torch.zeros(4, 64, device="cuda"), torch.zeros(4, device="cuda")
    S = ro.rowops_sample
    for call in (lambda: S(x, u, temperature=-1.0), lambda: S(x, u, top_k=-1), lambda: S(x, u, top_p=-0.5),
                 lambda: S(x, u, min_p=1.5), lambda: S(torch.zeros(1, 327681, device="cuda"), u[:1])):
        with pytest.raises(ro.RowopsError):
            call()
    for call in (lambda: S(x, u[:3]), lambda: S(x, u.double()), lambda: S(x, u, temperature=u[:3]),
                 lambda: S(x, u, top_k=torch.zeros(4, dtype=torch.int64, device="cuda")), lambda: S(x, u, top_p=u.cpu()),
                 lambda: S(x, u, min_p=u.double()), lambda: S(x, u, token=torch.zeros(4, device="cuda")),
                 lambda: S(x, u, logprob=torch.zeros(3, device="cuda")), lambda: S(x.cpu(), u), lambda: S(x[0], u)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        S(x.half(), u)
    assert S(x[:0], u[:0]).shape == (0,)


def test_top_k_of_more_than_32_bits():
    x, u = place(rows(4, 300, 31), "f32"), uniform(4, 32)
    for k in (300, 2**31, 2**32 + 1, 2**63 - 1, 2**64 + 1):
        assert torch.equal(ro.rowops_sample(x, u, top_k=k), ro.rowops_sample(x, u))
    for k in (-1, -(2**32), -(2**64)):
        with pytest.raises(ro.RowopsError):
            ro.rowops_sample(x, u, top_k=k)
    with pytest.raises(TypeError):
        ro.rowops_sample(x, u, top_k=50.5)


@pytest.mark.parametrize("N", [3000, 70000])
@pytest.mark.parametrize("n", [1, 2, 100, 254, 255, 256, 257, 258, 1500])
@pytest.mark.parametrize("equal", [1, 3])
def test_cuts_among_values_close_together(n, equal, N):
    """n values within 2^-8 of one another, groups of `equal` the same, all others far below."""
    M = 6
    g = torch.Generator().manual_seed(33)
    x = -6 + 0.5 * torch.randn(M, N, generator=g)
    for i in range(M):
        x[i, torch.randperm(N, generator=g)[:n]] = 1 + torch.randperm(n, generator=g).div(equal, rounding_mode="floor") * 2.0**-20
    x, u = place(x, "f32"), uniform(M, 34)
    for k in sorted({1, (n + 1) // 2, max(1, n - 1), n, n + 1}):
        check(x, u, top_k=k)
        check(x, u, top_k=k, top_p=0.45)
    for p in (0.3, 0.999):
        check(x, u, top_p=p)
        check(x, u, top_p=p, top_k=n + 5, temperature=0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [40, 257, 5000, 70000])
def test_cuts_among_values_near_zero(dtype, N):
    """One large logit, the others so far below it that they share the place of zero, of both signs, and 0 itself."""
    x = rows(6, N, 35, 0.5)
    x[:, ::7] = 0
    x[:, 1::14] = -0.0
    x[:, 5] = 30000.0
    x, u = place(x, dtype), 1 - uniform(6, 36) * 2.0**-4
    for k in (2, N // 3, N // 2, N - 1):
        check(x, u, temperature=20000.0, top_k=k)
        check(x, u, temperature=20000.0, top_k=k, top_p=0.6)
    check(x, u, temperature=20000.0, top_p=0.9)
    check(x, u, temperature=1e6, top_p=0.37)
