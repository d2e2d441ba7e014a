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
