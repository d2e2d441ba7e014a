"""The 64-bit forms of the serving operators against what fixes them: torch's own e4m3
conversion, dense attention, and draws counted by hand."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as O


def test_e4m3_half_step_is_what_a_conversion_moves_by():
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.logspace(-12, 2.6, 20001, base=10)]).double()
    moved = (v.float().to(torch.float8_e4m3fn).double() - v).abs()
    half = torch.from_numpy(O.e4m3_half_step(v.numpy()))
    assert torch.all(moved <= half * (1 + 1e-6))
    exact = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    exact = exact[torch.isfinite(exact)].sort().values.unique()
    middle = (exact[1:] + exact[:-1]) / 2  # the farthest from any number
    assert torch.allclose((exact[1:] - exact[:-1]) / 2, torch.from_numpy(O.e4m3_half_step(middle.numpy())))


def test_scales_of_groups():
    y = np.array([[1.0, -4.0, 0.5, 0.25, 448.0], [0, 0, 0, 0, 0]])
    assert np.array_equal(O.quant_scales(y, 2), [[4 / 448, 0.5 / 448, 1.0], [2.0**-126] * 3])
    assert np.array_equal(O.quant_scales(y, 0), [[1.0], [2.0**-126]])


@pytest.mark.parametrize("window", [0, 5])
def test_paged_attention_is_dense_attention_of_the_pages_in_turn(window):
    g = torch.Generator().manual_seed(1)
    H, K, D, page, lengths = 6, 2, 8, 4, [11, 0, 3]
    k, v = (torch.randn(9, page, K, D, generator=g) for _ in range(2))
    q = torch.randn(3, H, D, generator=g)
    table = np.array([[4, 0, 7], [1, 1, 1], [8, -1, -1]])
    out, lse, _, _ = O.paged_attention(q.numpy(), k.numpy(), v.numpy(), table, lengths, 0.3, window)
    for b, n in enumerate(lengths):
        if n == 0:
            assert np.all(out[b] == 0) and np.all(lse[b] == -np.inf)
            continue
        kk, vv = (c[table[b]].reshape(-1, K, D)[:n].double() for c in (k, v))
        if window:
            kk, vv = kk[-window:], vv[-window:]
        s = torch.einsum("hd,nhd->hn", q[b].double(), kk.repeat_interleave(H // K, dim=1)) * 0.3
        want = torch.einsum("hn,nhd->hd", torch.softmax(s, dim=1), vv.repeat_interleave(H // K, dim=1))
        assert np.allclose(out[b], want) and np.allclose(lse[b], torch.logsumexp(s, dim=1))


def test_paged_attention_of_bad_pages_and_lengths_is_not_a_number():
    k = np.ones((2, 4, 1, 2))
    out, lse, _, _ = O.paged_attention(np.ones((3, 1, 2)), k, k, np.array([[0, 2], [0, -1], [1, 0]]), [8, 4, 9], 1.0)
    assert np.isnan(out[0]).all() and np.all(out[1] == 1) and np.isnan(out[2]).all() and np.isnan(lse[[0, 2]]).all()


def test_sampling_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))  # of 8
    draw = lambda u, **k: O.sample_row(x, u, **k)[0]
    assert [draw(u) for u in (0, 0.12, 0.13, 0.62, 0.63, 0.87, 0.88, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [draw(u, top_k=2) for u in (0, 0.66, 0.67, 0.99)] == [1, 1, 2, 2]
    assert [draw(u, top_k=3) for u in (0.1, 0.9)] == [0, 2]  # of the equal ones the first
    assert [draw(u, top_p=0.49) for u in (0, 0.99)] == [1, 1] and draw(0.99, top_p=0.51) == 2
    assert draw(0.99, top_p=0.8) == 2 and draw(0.1, top_p=0.8) == 0  # 4 + 2 of 8 do not reach it, and one more
    assert draw(0.99, min_p=0.3) == 2 and draw(0.99, min_p=0.6) == 1
    assert draw(0.5, temperature=0) == 1
    token, lp, margin = O.sample_row(x, 0.3, top_k=2)
    assert token == 1 and math.isclose(lp, math.log(4 / 6)) and margin > 0.01
    assert O.sample_row(np.array([0.0, np.nan]), 0.5)[0] == -1 and O.sample_row(np.full(3, -np.inf), 0.5)[0] == -1
    assert O.sample_row(np.array([np.inf, 0, np.inf]), 0.6)[0] == 2
