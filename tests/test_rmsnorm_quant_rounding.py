"""What RMSNorm with an 8-bit result rounds: where the scale is above its least, y / scale is
448 s w / max |s w|, without the root. The kernels have s w (one rounding, and one in the maximum), the scale (the product
with the root, that with 1 / 448, and 1 / 448 itself: three), its reciprocal (one unit in the last place, two
roundings' worth), the two factors' product and the quotient (one each): 9 * 2^-24 of it at most. So q is the
nearest e4m3 number wherever the quotient is farther than that from the middle of two, and one of the two there."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import gpu_util as gu
from tests.test_parity_rmsnorm_quant import TYPES, place

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 64, 96])
@pytest.mark.parametrize("M,N,pad,offset", [(4, 4096, 0, 0), (3000, 2048, 0, 0), (900, 8192, 0, 0), (900, 4099, 3, 0), (900, 2050, 0, 0),
                                            (900, 1000, 0, 1), (9, 40000, 0, 0)])
def test_the_nearest_number(dtype, group, M, N, pad, offset):
    g = torch.Generator().manual_seed(N)
    x = place(torch.randn(M, N, generator=g), dtype, pad, offset)
    w = (1 + 0.2 * torch.randn(N, generator=g)).to("cuda", TYPES[dtype])
    q, scales, _ = ro.rowops_rmsnorm_quant(x, None, w, 1e-5, group)
    again, scales2, _ = ro.rowops_rmsnorm_quant(x, None, w, 1e-5, group)
    assert torch.equal(q.view(torch.uint8), again.view(torch.uint8)) and torch.equal(scales, scales2)
    p = x.double() * w.double()  # exact
    column = torch.arange(N, device="cuda") // (group or N)
    top = torch.zeros(M, int(column[-1]) + 1, dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, column.expand(M, N), p.abs(), "amax")
    v = 448 * p / top[:, column]
    numbers = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    numbers = numbers[torch.isfinite(numbers)].unique()
    middles = (numbers[1:] + numbers[:-1]) / 2
    off = v.abs() * (9 * 2.0**-24 * (1 + 1e-5))
    n = q.double()
    # the numbers that a value within `off` of v is rounded to, a middle to either
    assert torch.all(n >= numbers[torch.searchsorted(middles, v - off)])
    assert torch.all(n <= numbers[torch.searchsorted(middles, v + off, right=True)])
