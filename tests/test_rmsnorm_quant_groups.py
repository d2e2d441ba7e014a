"""GPU parity of RMSNorm with an 8-bit result for groups that span warps: their maxima meet in shared
memory, in three arrays taken in turn by rows, one set a team of threads. Rows many enough that every
team takes several, their sizes thousands of times apart in turn, so that a maximum left from an earlier row would show
in the scales. Bounds as in test_parity_rmsnorm_quant, here against torch in 64 bits."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import gpu_util as gu
from tests.test_parity_rmsnorm_quant import TYPES, place, relative

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


def hold(q, scales, s, w, group, eps=1e-5):
    M, N = s.shape
    y = s.double() / (s.double().square().mean(dim=1, keepdim=True) + eps).sqrt() * w.double()
    column = torch.arange(N, device="cuda") // group
    top = torch.zeros(M, -(-N // group), dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, column.expand(M, N), y.abs(), "amax")
    want = (top / 448.0).clamp(min=2.0**-126)
    assert scales.shape == want.shape
    off = (scales.double() - want).abs() / want
    assert float(off.max()) <= relative(N), f"scales off by {float(off.max()):.3g} at {divmod(int(off.argmax()), want.shape[1])}"
    v = y / want[:, column]
    half = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0**-6))) - 4)
    over = (q.double() - v).abs() - half - 2 * relative(N) * v.abs()
    assert float(over.max()) <= 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (5, 0), (6, 2)])
@pytest.mark.parametrize("M,N", [(20001, 640), (7001, 2048), (2001, 8191), (1201, 16000), (6001, 333)])
def test_rows_in_turn(dtype, residual, pad, offset, M, N):
    g = torch.Generator(device="cuda").manual_seed(M)
    # 2^12, 2^-8, 1, 2^6, 2^-12 times as large, in turn; groups of a row 1, 2^-5, 2^4 times
    size = torch.exp2(torch.tensor([12.0, -8.0, 0.0, 6.0, -12.0], device="cuda"))[torch.arange(M, device="cuda") % 5]
    within = torch.exp2(torch.tensor([0.0, -5.0, 4.0], device="cuda"))[torch.arange(N, device="cuda") // 96 % 3]

    def rows(factor):
        return place(factor * size[:, None] * within * torch.randn(M, N, generator=g, device="cuda"), dtype, pad, offset)

    x, r = rows(1.0), rows(2.0) if residual else None
    w = (1 + 0.2 * torch.randn(N, generator=g, device="cuda")).to(TYPES[dtype])
    for group in (96, 160, 256, 512):
        q, scales, s = ro.rowops_rmsnorm_quant(x, r, w, 1e-5, group)
        if residual:
            assert torch.equal(s, (x.float() + r.float()).to(x.dtype))
        hold(q, scales, s if residual else x, w, group)
        again, scales2, _ = ro.rowops_rmsnorm_quant(x, r, w, 1e-5, group)
        assert torch.equal(q.view(torch.uint8), again.view(torch.uint8)) and torch.equal(scales, scales2)
