"""Sampling at the ends of its ranges, against the 64-bit form; bounds as in test_parity_sample."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import gpu_util as gu
from tests.test_parity_sample import check, place, rows, uniform

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


@pytest.mark.parametrize("N", [3, 500, 20000])
@pytest.mark.parametrize("temperature", [2.0**-149, 1e-40, 4e-39, 2.0**-126, 2e-38, 1e-37])
def test_subnormal_temperatures(N, temperature):
    """Logits of a temperature's size: those below 2^-126 draw as 2^-126 does."""
    x = (rows(16, N, 41).double() * 2.0**-125).float()  # (subnormal for the most part)
    x, u = place(x, "f32"), uniform(16, 42)
    at = max(temperature, 2.0**-126)
    knobs = [{}, dict(top_k=2), dict(top_p=0.7), dict(min_p=0.2), dict(top_k=40, top_p=0.9, min_p=0.01)]
    for k in knobs:
        token, logprob = torch.empty(16, dtype=torch.int64, device="cuda"), torch.empty(16, device="cuda")
        ro.rowops_sample(x, u, temperature=temperature, **k, token=token, logprob=logprob)
        lp = torch.empty(16, device="cuda")
        assert torch.equal(token, ro.rowops_sample(x, u, temperature=at, **k, logprob=lp)) and torch.equal(logprob, lp)
        each = torch.full((16,), temperature, device="cuda")
        assert torch.equal(token, ro.rowops_sample(x, u, temperature=each, **k))
        assert torch.equal(token, check(x, u, temperature=at, **k))


def test_equal_maxima_at_a_subnormal_temperature():
    x = torch.zeros(8, 100, device="cuda")
    x[:, ::25] = 1.0
    u = (torch.arange(8, dtype=torch.float32) / 8).cuda()
    want = 25 * (torch.arange(8, device="cuda") // 2)
    for temperature in (2.0**-149, 1e-39):
        assert torch.equal(ro.rowops_sample(x, u, temperature=temperature), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [500, 70000])
@pytest.mark.parametrize("knobs", [{}, dict(top_k=400), dict(min_p=1e-16), dict(temperature=torch.ones(6))])
def test_the_least_weight_that_is_drawn(dtype, N, knobs):
    """u = 0 draws the first column that has a weight: of 2^-45 of the maximum's at least."""
    x = torch.full((6, N), -200.0)
    x[:, 300:303] = 0.0
    x[:3, 7], x[3:, 7] = -30.75, -31.5  # 2^-44.4, 2^-45.4
    knobs = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in knobs.items()}
    logprob = torch.empty(6, device="cuda")
    got = ro.rowops_sample(place(x, dtype), torch.zeros(6, device="cuda"), **knobs, logprob=logprob)
    assert got.tolist() == [7] * 3 + [300] * 3
    want = torch.tensor([-30.75] * 3 + [0.0] * 3) - torch.log(torch.tensor(3.0))
    assert torch.all((logprob.cpu() - want).abs() <= 2.0**-22 * want.abs() + 2.0**-28)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("depth", [10, 20, 30, 40])
def test_small_weights_are_right_to_their_bound(dtype, depth):
    """Among n columns of 2^-depth each beside one maximum, the draw's border lies where the sum of the small weights says:
    off by n (2^-29 of a weight, and 2^-45)."""
    N = 60000
    x = torch.full((1, N), -depth * 0.6931471805599453)
    x[0, N - 1] = 0.0
    x = place(x, dtype)
    w = torch.exp(x[0, 0].double())
    mass = float(w) * (N - 1)
    bound = (N - 1) * (float(w) * 2.0**-29 + 2.0**-45) / (1 + mass) + 2.0**-24  # (u itself, at most 1 + 2^-24 of its value)
    part = mass / (1 + mass)
    u = torch.tensor([max(part - bound, 0.0), min(part + bound, 1 - 2.0**-24)], dtype=torch.float64).float().cuda()
    last = ro.rowops_sample(x.expand(2, -1).contiguous(), u).tolist()
    assert last[1] == N - 1 and (last[0] < N - 1 or float(u[0]) == 0)
