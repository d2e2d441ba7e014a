"""A streamed group norm whose results never come stops after one wait a CTA.

No GPU fault is involved: ROWOPS_TEST_STALL_ROW withholds a sample's results and
ROWOPS_WAIT_LIMIT_NS shortens the waits; the kernel records the timeout."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TIMEOUT = 5
LIMIT_MS = 50


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B", [1, 2])
def test_a_wait_that_runs_out_ends_the_call(B, backward, monkeypatch):
    """Ten or more chunks for each CTA, one an SM (403 MB in chunks of 192 KB; in the
    backward pass twice that, of 512 KB): one wait after the other for the
    withheld sample's would take ten limits or, of two samples, five. A CTA waits
    once, and no wait begins more than one limit after the first: two limits, and
    the sums before them (a millisecond)."""
    S, C, G = 1536 * 1024 // B, 128, 32
    x = torch.randn(B, S, C, device="cuda", dtype=torch.bfloat16)
    stats = torch.empty(B, G, 2, device="cuda")
    monkeypatch.setenv("ROWOPS_GROUPNORM", "stream")
    monkeypatch.setenv("ROWOPS_CTAS_PER_SM", "1")

    def call():
        if backward:
            return ro.rowops_groupnorm_act_backward(x, x, stats, G)
        return (ro.rowops_groupnorm_act(x, G, stats=stats),)

    ro.rowops_groupnorm_act(x, G, stats=stats)
    clean = call()
    assert ro.rowops_device_status() == 0
    monkeypatch.setenv("ROWOPS_WAIT_LIMIT_NS", str(LIMIT_MS * 1000000))
    monkeypatch.setenv("ROWOPS_TEST_STALL_ROW", "5")
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    call()
    t1.record()
    assert ro.rowops_device_status() == TIMEOUT
    assert LIMIT_MS <= t0.elapsed_time(t1) <= 3 * LIMIT_MS
    monkeypatch.delenv("ROWOPS_TEST_STALL_ROW")
    for u, v in zip(call(), clean):
        assert torch.equal(u, v)
    assert ro.rowops_device_status() == 0
