"""RMSNorm with an 8-bit result at the ends of what its products s w may be: up to 2^128 they are right, one
beyond is its group's alone, and below 2^-126 a product is right to 2^-150. So there y is right to inv 2^-150
beside the bounds of test_parity_rmsnorm_quant (inv = 1 / sqrt(mean s^2 + eps)), a scale to that / 448, and y / scale to
twice that / scale (once for y, once for the scale at |y / scale| = 448), and twice again where the scale is up to
half off."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import serving as O
from tests import _compare as C
from tests import gpu_util as gu
from tests.test_parity_rmsnorm_quant import TYPES, hold, place, relative

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

SHAPES = [(512, 0), (2048, 0), (1022, 0), (333, 3), (40000, 0)]  # 16-byte vectors, pieces of 4 and 2, and rows in a loop
GROUPS = [0, 32, 96, 128, 512]


def rows(M, N, dtype, size, pad, seed):
    g = torch.Generator().manual_seed(seed)
    return place(size * torch.randn(M, N, generator=g).clamp(-4, 4), dtype, pad)


def weights(N, dtype, size, seed):
    g = torch.Generator().manual_seed(seed)
    return (size * (0.5 + torch.rand(N, generator=g))).to("cuda", TYPES[dtype])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size,eps", [(1.0, 1e-5), (1e15, 1e-5), (1e-15, 0.0)])
@pytest.mark.parametrize("N,pad", SHAPES)
def test_the_largest_products(dtype, size, eps, N, pad):
    x = rows(9, N, dtype, size, pad, 1)
    w = weights(N, dtype, 1.0, 2)
    largest = float((x.double() * w.double()).abs().max())
    w = (w.double() * min(2.0**127.9 / largest, 2.0**125)).to(w.dtype)  # (the product, and w itself, up to 2^128)
    assert float((x.double() * w.double()).abs().max()) < 2.0**128 and torch.isfinite(w).all()
    for group in GROUPS:
        q, scales, _ = ro.rowops_rmsnorm_quant(x, None, w, eps, group)
        hold(q, scales, C.to_f64(x), C.to_f64(w), group, eps)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,pad", SHAPES)
def test_a_product_beyond_is_its_groups_alone(dtype, N, pad):
    x = rows(700 if N < 4096 else 9, N, dtype, 1e15, pad, 3)
    w = weights(N, dtype, 1.0, 4)
    x[:, 200] = 2.0**50
    fine = {group: ro.rowops_rmsnorm_quant(x, None, w, 1e-5, group) for group in GROUPS[1:]}
    w[200] = 2.0**80
    for group in GROUPS[1:]:
        q, scales, _ = ro.rowops_rmsnorm_quant(x, None, w, 1e-5, group)
        if group >= N:
            assert torch.isinf(scales).all() and torch.isnan(q[:, 200].float()).all()
            continue
        g = 200 // group
        assert torch.isinf(scales[:, g]).all() and torch.isnan(q[:, 200].float()).all()
        others = torch.arange(scales.shape[1], device="cuda") != g
        assert torch.equal(scales[:, others], fine[group][1][:, others])
        columns = torch.arange(N, device="cuda") // group != g
        assert torch.equal(q.view(torch.uint8)[:, columns], fine[group][0].view(torch.uint8)[:, columns])
        rest = ~columns
        rest[200] = False
        assert torch.all(q.float()[:, rest] == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size,weight,eps", [(1e-15, 1e-27, 0.0), (1e-10, 1e-35, 1e-20), (1.0, 1e-38, 1e-5), (1e-17, 1e-30, 0.0)])
@pytest.mark.parametrize("N,pad", SHAPES)
def test_the_smallest_products(dtype, size, weight, eps, N, pad):
    x, w = rows(9, N, dtype, size, pad, 5), weights(N, dtype, weight, 6)
    s, f = C.to_f64(x), C.to_f64(w)
    lost = 2.0**-150 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    y = O.rmsnorm(s, f, eps)
    for group in GROUPS:
        q, scales, _ = ro.rowops_rmsnorm_quant(x, None, w, eps, group)
        want = O.quant_scales(y, group)
        off = np.abs(scales.double().cpu().numpy() - want)
        assert np.all(off <= relative(N) * want + lost / 448 * (1 + 1e-5) + 2.0**-149)
        each = np.repeat(want, group or N, axis=1)[:, :N]
        v, n = y / each, q.float().cpu().numpy().astype(np.float64)
        beside = 4 * lost / each  # the product's and the scale's, this less than half of the scale; else at most 448
        assert np.all(np.abs(n - v) <= O.e4m3_half_step(np.abs(v) + beside) + 2 * relative(N) * np.abs(v) + beside)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,pad", SHAPES)
def test_a_product_and_the_sum_of_squares_beyond(dtype, N, pad):
    """1 / root is 0: finite products give 0, as in rowops_rmsnorm, and a group with an infinite one is not a number."""
    x, w = rows(9, N, dtype, 1.0, pad, 7), weights(N, dtype, 1.0, 8)
    x[:, 200], w[200] = 1e25, 1e25
    for group in GROUPS:
        q, scales, _ = ro.rowops_rmsnorm_quant(x, None, w, 1e-5, group)
        g = torch.arange(scales.shape[1], device="cuda") == (200 // group if group else 0)
        columns = torch.arange(N, device="cuda") // (group or N) == (200 // group if group else 0)
        assert torch.isnan(scales[:, g]).all() and torch.isnan(q.float()[:, columns]).all()
        assert torch.all(scales[:, ~g] == 2.0**-126) and torch.all(q.float()[:, ~columns] == 0)
