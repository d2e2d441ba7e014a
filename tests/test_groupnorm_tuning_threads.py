"""Group norm called in one thread while another changes the library's knobs: a
call checks the workspace of the form that it launches. (The form that streams
needs one; the form that holds its slabs needs none forward.)"""
import os
import threading

import pytest
import torch

import row_wise_reduction_gb300 as ro
from row_wise_reduction_gb300.rowops import library
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

OK, WORKSPACE = 0, 3


def test_the_workspace_checked_is_that_of_the_form_launched(monkeypatch):
    B, S, C, G = 2, 64, 64, 4
    x = torch.randn(B, S, C, device="cuda")
    stats = torch.empty(B, G, 2, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    monkeypatch.setenv("ROWOPS_GROUPNORM", "fused")
    want = ro.rowops_groupnorm_act(x, G, stats=stats)
    wants = ro.rowops_groupnorm_act_backward(x, x, stats, G)
    L, stream = library(), torch.cuda.current_stream().cuda_stream
    held = L.rowops_groupnorm_act_backward_workspace_bytes(B, S, C, G, 0)
    ws = torch.empty(held, dtype=torch.uint8, device="cuda")
    done = threading.Event()

    def turn():
        while not done.is_set():
            for form in ("stream", "fused"):
                os.environ["ROWOPS_GROUPNORM"] = form
                ro.rowops_reload_tuning()

    t = threading.Thread(target=turn)
    t.start()
    seen = set()
    try:
        for _ in range(4000):
            seen.add(L.rowops_groupnorm_act(x.data_ptr(), y.data_ptr(), None, None, 1e-5, B, S, C, G, C, 1, None, 0,
                                            None, 0, stream))
            seen.add(L.rowops_groupnorm_act_backward(
                x.data_ptr(), x.data_ptr(), None, None, stats.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
                B, S, C, G, C, 1, 0, ws.data_ptr(), held, stream))
    finally:
        done.set()
        t.join()
    torch.cuda.synchronize()
    assert seen <= {OK, WORKSPACE} and OK in seen
    assert torch.equal(y, want)
    for got, ref in zip((dx, dw, db), wants):
        assert torch.equal(got, ref)
