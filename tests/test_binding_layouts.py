"""Layouts of given outputs at the ends: no rows at all, and a single row."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

N = 24


@pytest.mark.parametrize("op", [ro.rowops_softmax, ro.rowops_layernorm_gelu, ro.rowops_layernorm_gelu_erf,
                                ro.rowops_bias_dropout_residual])
def test_no_rows_into_a_spread_output(op):
    """Nothing is written, so any columns do (as with a given y of no rows ever)."""
    x = torch.empty(0, N, device="cuda")
    y = torch.empty(0, 2 * N, device="cuda")[:, ::2]
    assert y.stride(1) == 2
    assert op(x, y=y) is y


def test_no_rows_of_a_spread_residual():
    x = torch.empty(0, N, device="cuda")
    assert ro.rowops_bias_dropout_residual(x, torch.empty(0, 2 * N, device="cuda")[:, ::2]).shape == (0, N)


CALLS = {
    "online_softmax y": lambda x, t: ro.rowops_online_softmax(x, t),
    "online_softmax_noalloc y": lambda x, t: ro.rowops_online_softmax_noalloc(x, t),
    "softmax_causal y": lambda x, t: ro.rowops_softmax_causal(x, y=t),
    "backward dy": lambda x, t: ro.rowops_layernorm_gelu_backward(x, t),
    "backward dx": lambda x, t: ro.rowops_layernorm_gelu_backward(x, x, dx=t),
    "gelu residual": lambda x, t: ro.rowops_bias_residual_gelu(x, t),
    "gelu y": lambda x, t: ro.rowops_bias_residual_gelu(x, y=t),
    "rmsnorm y": lambda x, t: ro.rowops_rmsnorm(x, y=t),
    "fused rmsnorm residual": lambda x, t: ro.rowops_fused_residual_rmsnorm(x, t),
    "fused rmsnorm y": lambda x, t: ro.rowops_fused_residual_rmsnorm(x, x, y=t),
    "fused rmsnorm residual_out": lambda x, t: ro.rowops_fused_residual_rmsnorm(x, x, residual_out=t),
}


@pytest.mark.parametrize("call", CALLS)
def test_one_row_of_spread_columns_is_refused(call):
    """A single row has no row stride to compare, but its columns must be
    neighbours: the kernels write and read them as such."""
    x = torch.ones(1, N, device="cuda")
    with pytest.raises(ValueError):
        CALLS[call](x, torch.zeros(1, 2 * N, device="cuda")[:, ::2])
    far = torch.as_strided(torch.zeros(N, device="cuda"), (1, N), (1000, 1))  # its stride leads nowhere
    CALLS[call](x, far)
    torch.cuda.synchronize()
