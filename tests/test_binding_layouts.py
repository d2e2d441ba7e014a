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
