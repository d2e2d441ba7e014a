"""The serving operators where offsets pass 2^31 elements: normalised rows there are right, and
what pages and logits there give is what they give in a small tensor."""
import pytest
import torch

import row_wise_reduction_gb300 as ro
from tests import _compare as C
from tests import gpu_util as gu
from tests.test_parity_rmsnorm_quant import hold

pytestmark = [pytest.mark.gpu, gu.requires_gpu]


@pytest.mark.parametrize("N", [8192, 8191])
def test_rmsnorm_quant(N):
    M = (1 << 31) // N + 40
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    x[-64:] = torch.randn(64, N, device="cuda")
    q, s, out = ro.rowops_rmsnorm_quant(x, x, None, 1e-5, 128)
    # few rows are summed in another order than many: the rows are held to the 64-bit form
    hold(q[-64:], s[-64:], C.to_f64(out[-64:]), None, 128)
    assert torch.equal(out[-64:], x[-64:] + x[-64:])
    assert torch.all(q[: 1 << 17].view(torch.uint8) == 0)


@pytest.mark.parametrize("width", [40, 60000])
@pytest.mark.parametrize("layout", ["slots", "heads"])
def test_paged_attention(width, layout):
    pages, page, K, D, H = 140000, 16, 8, 128, 16
    shape = (pages, page, K, D) if layout == "slots" else (pages, K, page, D)
    k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if layout == "heads":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    far = torch.arange(pages - 40, pages, device="cuda").flip(0)
    near = torch.arange(40, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for c in (k, v):
        c[far] = torch.randn(40, page, K, D, device="cuda", generator=g).bfloat16()
        c[near] = c[far]
    q = torch.randn(1, H, D, device="cuda", generator=g).bfloat16().expand(2, H, D).contiguous()
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0, :40], table[1, :40] = far.int(), near.int()
    n = torch.tensor([639, 639], dtype=torch.int32, device="cuda")
    out = ro.rowops_paged_attention(q[1:], k, v, table[1:], n[1:])
    assert torch.equal(ro.rowops_paged_attention(q[:1], k, v, table[:1], n[:1]), out)
    both = ro.rowops_paged_attention(q, k, v, table, n)
    assert torch.allclose(both.float(), out.float().expand(2, H, D), rtol=2.0**-7, atol=1e-5)
    assert out.float().abs().max() > 0.1


@pytest.mark.parametrize("N", [131072, 131071])
def test_sample(N):
    M = (1 << 31) // N + 10
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    x[-16:] = 3 * torch.randn(16, N, device="cuda")
    u = torch.rand(M, device="cuda")
    t = ro.rowops_sample(x, u, top_k=1000, top_p=0.9)
    assert torch.equal(t[-16:], ro.rowops_sample(x[-16:].clone(), u[-16:], top_k=1000, top_p=0.9))
    assert torch.all(t[:-16] < 1000)  # equal logits: the first 900
