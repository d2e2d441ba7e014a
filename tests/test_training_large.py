"""The training operators on tensors of more than 2^31 elements: their last rows
against the 64-bit forms (bounds as in the operators' own tests)."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import training as O
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N", [4096, 4099])  # vectors; rows at changing offsets
def test_dropout(N):
    M = 2**31 // N + 1001
    x = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    b = torch.full((N,), 0.5, dtype=torch.bfloat16, device="cuda")
    y = ro.rowops_bias_dropout_residual(x, None, b, 0.5, 3, 1)
    keep = O.dropout_keep(np.arange(M - 3, M), N, 0.5, 3, 1)
    assert np.array_equal(y[-3:].float().cpu().numpy(), 3.0 * keep)
    dx, db = ro.rowops_bias_dropout_residual_backward(x, 0.5, 3, 1)
    assert np.array_equal(dx[-3:].float().cpu().numpy(), 2.0 * keep)
    kept = sum((dx[i:i + 65536] != 0).sum(dim=0) for i in range(0, M, 65536))
    assert torch.equal(db, 2.0 * kept.float())  # whole numbers below 2^24: exact
    del x, y, dx


def test_groupnorm():
    B, C, G = 2, 512, 32
    S = 2**31 // (B * C) + 77
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(B, S, C, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(B, S, C, generator=g, device="cuda", dtype=torch.bfloat16)
    stats = torch.empty(B, G, 2, device="cuda")
    y = ro.rowops_groupnorm_act(x, G, act="none", stats=stats)
    dx, dw, db = ro.rowops_groupnorm_act_backward(x, dy, stats, G, act="none")
    rdw = rdb = 0
    for n in range(B):
        v, d = x[n].double().view(S, G, -1), dy[n].double().view(S, G, -1)
        mean, rstd = v.mean(dim=(0, 2)), 1 / (v.var(dim=(0, 2), correction=0) + 1e-5).sqrt()
        xh = (v - mean[:, None]) * rstd[:, None]
        del v
        tail = xh[-5:].reshape(5, C)
        assert torch.all((y[n, -5:] - tail).abs() <= 1e-5 * tail.abs().clamp(min=1) + 2.0**-8 * tail.abs())
        c1, c2 = d.mean(dim=(0, 2)), (d * xh).mean(dim=(0, 2))
        r = (rstd[:, None] * (d[-5:] - c1[:, None] - xh[-5:] * c2[:, None])).reshape(5, C)
        size = (rstd[:, None] * (d[-5:].abs() + 1 + xh[-5:].abs())).reshape(5, C)
        assert torch.all((dx[n, -5:] - r).abs() <= 2e-5 * size + 2.0**-8 * r.abs())
        rdw = rdw + (d * xh).sum(dim=0).reshape(-1)
        rdb = rdb + d.sum(dim=0).reshape(-1)
        del xh, d
    # means of |dy| and |dy xh| are 0.8 and 0.64
    assert torch.all((db - rdb).abs() <= 2e-5 * 0.8 * B * S) and torch.all((dw - rdw).abs() <= 2e-5 * 0.64 * B * S)
    del x, dy, y, dx


def test_router():
    E, K = 256, 2
    T = 2**31 // E + 4097
    g = torch.Generator(device="cuda").manual_seed(6)
    logits = torch.randn(T, E, generator=g, device="cuda", dtype=torch.bfloat16)
    experts = torch.randint(0, E, (T, K), generator=g, device="cuda")
    loss, counts = ro.rowops_router_balance_loss(logits, experts, 0.5)
    want = torch.bincount(experts.reshape(-1), minlength=E)
    assert torch.equal(counts[:E], want) and int(counts[E]) == T
    P = sum(torch.softmax(logits[i:i + 2**20].double(), dim=1).sum(dim=0) for i in range(0, T, 2**20))
    ref = float(0.5 * E * (want / (T * K) * P / T).sum())
    assert abs(float(loss) - ref) <= 1.5e-5 * ref
    d = ro.rowops_router_balance_loss_backward(logits, counts, K, torch.full((1,), 1e6, device="cuda"), 0.5)
    rd, size = O.router_balance_loss_backward(logits[-9:].double().cpu().numpy(), counts.cpu().numpy(), K, 1e6, 0.5)
    assert np.all(np.abs(d[-9:].double().cpu().numpy() - rd) <= 1e-5 * size + 2.0**-8 * np.abs(rd) + 2.0**-120)
