"""GPU parity of the attention of one token over a paged cache with its 64-bit form.
With steps = max_j |scale| sum_d |q_d k_jd|, a score is off by at most (D + 2) 2^-24
steps; exp of the difference to the maximum by 2^-22 and 2^-23 of the difference, at
most 2 steps, more; sums over n positions by n 2^-24 at worst. So out is off by at most
rel sum p |v| with rel = 2 ((D + 6) 2^-24 steps + 2^-22 + n 2^-24), lse by rel and
its own rounding; bf16 adds 2^-8 |out| (its one rounding), and 2^-16 sum p |v| for
weights that enter the products as two bf16 numbers."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import serving as O
from tests import _compare as C
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def problem(lengths, H, K, D, page, dtype, layout="slots", seed=1, width=None, qpad=0, wide=0):
    """q, k, v, table, lengths: pages anywhere in the pool, NaN in every slot past a
    sequence's end and in every page of none, -7 where the table has no page."""
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    need = [-(-max(n, 0) // page) for n in lengths]
    width = max(need + [1]) if width is None else width
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=g)
    shape = {"slots": (pool, page, K, D + wide), "heads": (pool, K, page, D + wide)}[layout]
    caches = []
    for _ in range(2):
        c = torch.randn(shape, generator=g).to(TYPES[dtype])
        caches.append((c if layout == "slots" else c.transpose(1, 2))[..., :D])
    table = torch.full((B, width), -7, dtype=torch.int32)
    at = 0
    used = torch.zeros(pool, page, dtype=torch.bool)
    for b, n in enumerate(lengths):
        mine = order[at:at + need[b]]
        table[b, : need[b]] = mine.int()
        at += need[b]
        for i, p in enumerate(mine.tolist()):
            used[p, : max(0, min(page, n - i * page))] = True
    for c in caches:
        c[~used] = float("nan")
    q = torch.randn(B, H * D + qpad, generator=g).to(TYPES[dtype])
    # (Tensor.to keeps the caches' strides)
    k, v = (torch.empty_strided(c.shape, c.stride(), dtype=c.dtype, device="cuda").copy_(c) for c in caches)
    q = q.cuda()[:, : H * D].unflatten(1, (H, D))
    return q, k, v, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda")


def check(lengths, H, K, D, page, dtype, window=0, scale=None, **more):
    q, k, v, table, n = problem(lengths, H, K, D, page, dtype, **more)
    B = len(lengths)
    out = torch.full((B + 2, H, D), 3.0, dtype=q.dtype, device="cuda")
    lse = torch.full((B + 2, H), 3.0, device="cuda")
    got = ro.rowops_paged_attention(q, k, v, table, n, scale, window, out[1:-1], lse[1:-1])
    assert torch.all(out[0] == 3) and torch.all(out[-1] == 3) and torch.all(lse[0] == 3) and torch.all(lse[-1] == 3)
    hold(got, lse[1:-1], q, k, v, table, n, scale, window)
    return got, lse[1:-1], (q, k, v, table, n)


def hold(got, lse, q, k, v, table, n, scale=None, window=0):
    D = q.shape[2]
    dtype = "f32" if q.dtype == torch.float32 else "bf16"
    ref, rlse, size, steps = O.paged_attention(*(C.to_f64(t) for t in (q, k, v)), table.cpu().numpy(), n.cpu().numpy(),
                                               D**-0.5 if scale is None else scale, window)
    longest = max(1, min(int(n.max()), table.shape[1] * k.shape[1]))
    rel = 2 * ((D + 6) * 2.0**-24 * steps + 2.0**-22 + longest * 2.0**-24)
    tol = rel[..., None] * size + 2.0**-126
    if dtype == "bf16":
        tol = tol + 2.0**-8 * np.abs(ref) + 2.0**-16 * size
    g, gl = C.to_f64(got), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isnan(gl), np.isnan(rlse))
    fine = ~np.isnan(ref)
    err = np.abs(g - ref)
    assert np.all(err[fine] <= tol[fine]), f"off by {np.max((err / tol)[fine]):.3g} of what is allowed"
    empty = rlse == -np.inf
    assert np.all(gl[empty] == -np.inf) and np.all(g[empty] == 0)
    fine = np.isfinite(rlse)
    assert np.all(np.abs(gl[fine] - rlse[fine]) <= rel[fine] + 2.0**-22 * np.abs(rlse[fine]))


LINE = 100000  # a table this wide (most of it unused) makes it equal stretches of tiles, and parts


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1000, 4097])
def test_lengths(dtype, n):
    check([n], 8, 2, 64, 16, dtype)
    check([n], 8, 2, 64, 16, dtype, width=LINE)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 3, 8, 17, 32, 40, 63, 64, 72, 80, 96, 100, 112, 128, 160, 192, 200, 255, 256])
def test_head_dimensions(dtype, D):
    check([130, 1, 77], 6, 2, D, 16, dtype)
    check([130, 1, 77], 6, 2, D, 16, dtype, width=LINE)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,K", [(1, 1), (2, 1), (5, 5), (6, 2), (15, 3), (7, 1), (8, 1), (12, 1), (16, 1), (17, 1), (40, 2),
                                 (71, 1), (128, 8)])
def test_heads(dtype, H, K):
    check([200, 31], H, K, 64, 16, dtype)
    check([200, 31], H, K, 64, 16, dtype, width=LINE)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [1, 3, 8, 24, 32, 100, 128, 1000])
@pytest.mark.parametrize("layout", ["slots", "heads"])
def test_pages_and_layouts(dtype, page, layout):
    check([333, 5, 100], 8, 2, 64, page, dtype, layout=layout)
    check([333, 5, 100], 8, 2, 64, page, dtype, layout=layout, width=LINE)


@pytest.mark.parametrize("dtype", TYPES)
def test_empty_sequences_and_ragged_batches(dtype):
    for width in (50, LINE):
        check([0, 700, 0, 1, 64, 0], 8, 4, 64, 16, dtype, width=width)
        check([0, 0], 4, 4, 32, 8, dtype, width=width)
        check([-5, 20], 4, 4, 32, 8, dtype, width=width)
    check([(i * 37) % 301 for i in range(67)], 4, 2, 64, 16, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 299, 300, 10**9])
def test_windows(dtype, window):
    check([300, 64, 1, 0, 150], 8, 2, 64, 16, dtype, window=window)
    check([300, 64, 1, 0, 150] + [20] * 200, 8, 2, 64, 16, dtype, window=window, width=LINE)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,wide,qpad", [(64, 8, 8), (64, 3, 0), (80, 0, 3), (36, 4, 1), (128, 1, 0)])
def test_strides_and_alignment(dtype, D, wide, qpad):
    check([90, 200], 4, 2, D, 16, dtype, wide=wide, qpad=qpad)
    check([90, 200], 4, 2, D, 16, dtype, wide=wide, qpad=qpad, layout="heads")
    check([90, 200], 4, 2, D, 16, dtype, wide=wide, qpad=qpad, width=LINE)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
def test_scales(dtype, scale):
    check([150, 40], 4, 2, 32, 16, dtype, scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_long_sequence_and_many(dtype):
    check([20000], 4, 1, 64, 16, dtype)
    check([3000 - 11 * i for i in range(40)], 8, 8, 32, 32, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [16, 12])  # whole pieces of a page, and not
@pytest.mark.parametrize("more", [0, 200])  # few sequences, and enough for equal stretches
def test_pages_outside_the_pool_and_lengths_beyond_the_table(dtype, page, more):
    q, k, v, table, n = problem([100, 100, 100, 20, 100] + [10] * more, 8, 2, 64, page, dtype)
    lse = torch.empty(5 + more, 8, device="cuda")
    last = 99 // page
    table[1, 2] = -1
    table[2, last] = k.shape[0]
    table[3, 2] = 1 << 30  # not reached
    n[4] = table.shape[1] * page + 1
    out = ro.rowops_paged_attention(q, k, v, table, n, lse=lse)
    hold(out, lse, q, k, v, table, n)
    n[4] = 2**31 - 1
    out = ro.rowops_paged_attention(q, k, v, table, n, lse=lse)
    hold(out, lse, q, k, v, table, n)
    table[1, 2] = table[0, 0]
    n[1] = 40  # the bad page within a window's reach or not
    table[2, 0] = -9
    table[2, last] = table[0, 1]
    out = ro.rowops_paged_attention(q, k, v, table, n, None, 50, lse=lse)
    hold(out, lse, q, k, v, table, n, None, 50)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_not_a_number(dtype):
    q, k, v, table, n = problem([70, 70, 70], 4, 2, 32, 16, dtype)
    at = table[0].long()
    k[at[1], 3, 0] = float("nan")          # a NaN key: its heads alone
    v[table[1, 2].long(), 5, 1, 4] = float("inf")   # an infinite value: one column of its heads (infinite or NaN)
    out = ro.rowops_paged_attention(q, k, v, table, n)
    assert torch.isnan(out[0, :2]).all() and torch.isfinite(out[0, 2:]).all()
    assert not torch.isfinite(out[1, 2:, 4]).any() and torch.isfinite(out[1, :2]).all()
    assert torch.isfinite(out[1, 2:, :4]).all() and torch.isfinite(out[1, 2:, 5:]).all() and torch.isfinite(out[2]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_apart(dtype):
    """One key that takes everything, at the start, the middle and the end."""
    for where in (0, 150, 299):
        q, k, v, table, n = problem([300], 2, 1, 64, 16, dtype)
        k[table[0, where // 16].long(), where % 16, 0] = 40 * torch.sign(q[0, 0])
        lse = torch.empty(1, 2, device="cuda")
        hold(ro.rowops_paged_attention(q, k, v, table, n, lse=lse), lse, q, k, v, table, n)


@pytest.mark.parametrize("width", [57, 4000])  # one kernel; two, with a workspace
def test_repeatable_on_a_stream_and_in_a_replayed_graph(width):
    q, k, v, table, n = problem([500, 33, 900, 0], 8, 2, 128, 16, "bf16", width=width)
    out = ro.rowops_paged_attention(q, k, v, table, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = ro.rowops_paged_attention(q, k, v, table, n, stream=s)
    s.synchronize()
    assert torch.equal(out, again)
    need = ro.rowops_paged_attention_workspace_bytes(4, 8, 2, 128, 16, width, 0, q.dtype)
    assert (need > 0) == (width == 4000)
    ws = torch.full((max(need, 256),), 0xff, dtype=torch.uint8, device="cuda")  # its contents do not matter
    y, lse = torch.empty_like(out), torch.empty(4, 8, device="cuda")
    ro.rowops_paged_attention(q, k, v, table, n, out=y, lse=lse, workspace=ws)
    assert torch.equal(out, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ro.rowops_paged_attention(q, k, v, table, n, out=y, lse=lse, workspace=ws)
    for lengths in ([500, 33, 900, 0], [1, 40, 37, 0], [0, 48, 899, 0]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        m = torch.tensor([min(a, b) for a, b in zip(lengths, [500, 33, 900, 0])], dtype=torch.int32, device="cuda")
        n.copy_(m)
        ws.fill_(0x7f)
        g.replay()
        hold(y, lse, q, k, v, table, n)


def test_refusals():
    q, k, v, table, n = problem([20, 9], 4, 2, 32, 8, "f32")
    P = ro.rowops_paged_attention
    for call in (lambda: P(q[0], k, v, table, n), lambda: P(q, k[..., :16], v, table, n),
                 lambda: P(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), table, n),
                 lambda: P(q, k.bfloat16(), v, table, n), lambda: P(q, k, v, table[:1], n),
                 lambda: P(q, k, v, table, n[:1]), lambda: P(q, k, v, table.long(), n), lambda: P(q, k, v, table, n.long()),
                 lambda: P(q, k, v, table, n, out=torch.empty(2, 4, 33, device="cuda")),
                 lambda: P(q, k, v, table, n, lse=torch.empty(7, device="cuda")),
                 lambda: P(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, table, n),
                 lambda: P(q, k.cpu(), v, table, n), lambda: P(q.cpu(), k, v, table, n)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ro.RowopsError):
        P(q[:, :3].contiguous(), k, v, table, n)  # 3 heads over 2
    with pytest.raises(ro.RowopsError):
        P(q, k, v, table, n, window=-1)
    with pytest.raises(ro.RowopsError):
        P(q, k, v, table, n, scale=float("nan"))
    assert P(q[:0], k, v, table[:0], n[:0]).shape == (0, 4, 32)


def test_no_columns_are_refused():
    q, k, v, table, n = problem([20, 9], 4, 2, 32, 8, "f32")
    for heads in (1, 4):
        with pytest.raises((ro.RowopsError, ValueError)):
            ro.rowops_paged_attention(q[:, :heads, :0].contiguous(), k[:, :, :1, :0], v[:, :, :1, :0], table, n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, LINE])
def test_a_cache_without_pages(dtype, width):
    q, k, v, table, n = problem([20, 0], 4, 2, 32, 16, dtype, width=width)
    lse = torch.empty(2, 4, device="cuda")
    out = ro.rowops_paged_attention(q, k[:0], v[:0], table, n, lse=lse)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf"))
    none = ro.rowops_paged_attention(q, k, v, table[:, :0], n, lse=lse)  # and a table without columns
    assert torch.isnan(none[0]).all() and torch.all(none[1] == 0) and torch.all(lse[1] == -float("inf"))
