"""Streamed group norm: a sample's values do not depend on the samples beside it in
the batch, whose number changes the chunks that a sample is cut into, the order of
the work and whether a sample's sums are joined in one step or two."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,S,C,G", [(5, 20000, 64, 4), (3, 66000, 256, 8), (40, 1500, 96, 12), (9, 4099, 33, 3)])
def test_a_sample_alone_gives_what_it_gives_in_the_batch(B, S, C, G, dtype, monkeypatch):
    """Both are within the operator's bounds of the true values (statistics 4e-6 of
    the spread and 1e-5, values 1e-5 of max(1, |y|), gradients 2e-5 of their
    terms' magnitudes), so twice those apart at most, and in bf16 one rounding
    step of the result, 2^-7."""
    monkeypatch.setenv("ROWOPS_GROUPNORM", "stream")
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(B, S, C, generator=g, device="cuda").to(dtype)
    dy = torch.randn(B, S, C, generator=g, device="cuda").to(dtype)
    x[B // 2] *= 50  # unlike its neighbours
    x[-1] += 7
    u = 2.0**-7 if dtype is torch.bfloat16 else 0.0
    stats = torch.empty(B, G, 2, device="cuda")
    y = ro.rowops_groupnorm_act(x, G, stats=stats)
    dx, dw, db = ro.rowops_groupnorm_act_backward(x, dy, stats, G)
    sums = [torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(4)]
    for n in range(B):
        st = torch.empty(1, G, 2, device="cuda")
        one = ro.rowops_groupnorm_act(x[n:n + 1], G, stats=st)
        mean, rstd = stats[n, :, 0], stats[n, :, 1]
        assert torch.all((st[0, :, 0] - mean).abs() <= 8e-6 / rstd + 2.0**-22 * mean.abs())
        assert torch.all((st[0, :, 1] / rstd - 1).abs() <= 2e-5)
        top = torch.maximum(one.abs(), y[n:n + 1].abs()).float()
        assert torch.all((one.float() - y[n:n + 1].float()).abs() <= 2e-5 * top.clamp(min=1) + u * top)
        # the same statistics: the sums over the group, then, alone differ
        done, dw1, db1 = ro.rowops_groupnorm_act_backward(x[n:n + 1], dy[n:n + 1], stats[n:n + 1].contiguous(), G)
        xh = ((x[n].float().view(S, G, -1) - mean[:, None]) * rstd[:, None])
        d = dy[n].float().abs().view(S, G, -1)
        size = rstd[:, None] * (d + d.mean(dim=(0, 2))[:, None] + xh.abs() * (d * xh.abs()).mean(dim=(0, 2))[:, None])
        top = torch.maximum(done.abs(), dx[n:n + 1].abs()).float()
        assert torch.all((done.float() - dx[n:n + 1].float()).abs() <= 4e-5 * size.view(1, S, C) + u * top)
        for total, v in zip(sums, (dw1, db1, (d * xh.abs()).sum(dim=0).view(C), d.sum(dim=0).view(C))):
            total += v.double()
    assert torch.all((dw - sums[0]).abs() <= 4e-5 * sums[2]) and torch.all((db - sums[1]).abs() <= 4e-5 * sums[3])
