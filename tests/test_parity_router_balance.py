"""GPU parity of the router's balance loss and its gradient with the 64-bit
form. Counts are exact. Loss: probabilities to 1e-6 relative (exp2 and one
division), sums of positive terms, at most 256 in turn: 256 2^-24 = 1.5e-5
relative. Gradient: 1e-5 of the magnitudes it is the difference of (a softmax to
1e-6, a dot product of at most 32 terms a lane and five levels), in bf16 a
rounding, 2^-8, more; probabilities below 2^-126 flush to 0."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import training as O
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEF = 0.01


def make(T, E, K, dtype, pad=0, offset=0, seed=1, wide=True):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    base = torch.full((T * (E + pad) + offset + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    logits = torch.as_strided(base, (T, E), (E + pad, 1), offset)
    logits.copy_(v)
    experts = v.topk(K, dim=1).indices.to("cuda", torch.int64 if wide else torch.int32)
    return logits, experts


def check(T, E, K, dtype, mask=None, logits=None, experts=None, **how):
    made = make(T, E, K, dtype, **how)
    logits = made[0] if logits is None else logits
    experts = made[1] if experts is None else experts
    ln, en = logits.double().cpu().numpy(), experts.cpu().numpy()
    mn = None if mask is None else mask.cpu().numpy()
    loss, counts = ro.rowops_router_balance_loss(logits, experts, COEF, mask)
    rl, rc = O.router_balance_loss(ln, en, COEF, mn)
    assert counts.cpu().numpy().tolist() == rc.tolist()
    assert abs(float(loss) - rl) <= 1.5e-5 * abs(rl)
    dloss = torch.full((1,), 1.75, device="cuda")
    d, buf, inside = gu.guarded_like(logits, offset=how.get("offset", 0))
    ro.rowops_router_balance_loss_backward(logits, counts, K, dloss, COEF, mask, d)
    rd, size = O.router_balance_loss_backward(ln, rc, K, 1.75, COEF, mn)
    err = np.abs(d.double().cpu().numpy() - rd)
    tol = 1e-5 * size + 2.0**-120 + (2.0**-8 * np.abs(rd) if dtype == "bf16" else 0)
    assert np.all(err <= tol), f"off by {np.max(err / tol):.3g} of what is allowed"
    gu.assert_guard_untouched(buf, inside)
    return logits, experts, loss, counts, d


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,K", [(1, 1), (2, 1), (3, 2), (7, 2), (8, 2), (16, 4), (60, 6), (64, 8), (65, 3), (100, 8),
                                 (128, 8), (256, 8), (320, 2), (513, 9), (1000, 40), (1024, 64)])
def test_expert_counts(dtype, E, K):
    check(403, E, K, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 1000, 20011])
def test_token_counts(dtype, T):
    check(T, 64, 6, dtype)
    check(T, 10, 1, dtype, wide=False)


def test_many_tokens():
    check(100003, 128, 8, "f32")
    check(30001, 1024, 8, "bf16")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (8, 8), (5, 2)])
def test_strides_and_alignment(dtype, pad, offset):
    check(300, 64, 4, dtype, pad=pad, offset=offset)
    check(300, 20, 4, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,pad,offset", [(2, 0, 0), (6, 2, 2), (62, 0, 0), (92, 4, 0), (510, 0, 2), (1022, 0, 0),
                                          (1021, 0, 1), (33, 2, 0)])
def test_rows_of_short_words(dtype, E, pad, offset):
    """Rows that are no whole vectors, several of them a warp and ten a thread."""
    check(5003, E, min(E, 3), dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
@pytest.mark.parametrize("T", [50, 9000])
def test_padded_rows(kind, T):
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(2)) < 0.6).to("cuda", kind)
    logits, experts = make(T, 64, 4, "f32")
    off = mask == 0
    logits[off] = float("nan")  # not read
    experts[off] = 1 << 40
    clean = torch.where(off[:, None], torch.zeros_like(logits), logits)
    want = ro.rowops_router_balance_loss(clean, torch.where(off[:, None], 0, experts), COEF, mask)
    got = ro.rowops_router_balance_loss(logits, experts, COEF, mask)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d = ro.rowops_router_balance_loss_backward(logits, got[1], 4, torch.ones(1, device="cuda"), COEF, mask)
    assert torch.all(d[off] == 0) and torch.isfinite(d).all()
    check(T, 64, 4, "f32", mask=mask, logits=clean)


@pytest.mark.parametrize("T", [40, 9000])
def test_nobody_takes_part(T):
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    logits, experts = make(T, 64, 2, "f32")
    loss, counts = ro.rowops_router_balance_loss(logits, experts, COEF, mask)
    assert float(loss) == 0 and torch.all(counts == 0)
    d = ro.rowops_router_balance_loss_backward(logits, counts, 2, torch.ones(1, device="cuda"), COEF, mask)
    assert torch.all(d == 0)


def test_masked_experts_and_dead_rows():
    logits, experts = make(200, 24, 2, "f32")
    logits[:, 5] = float("-inf")
    logits[17] = float("-inf")  # a row without any expert
    logits[18, 1:] = torch.finfo(torch.float32).min
    *_, d = check(200, 24, 2, "f32", logits=logits, experts=experts)
    assert torch.all(d[:, 5] == 0) and torch.all(d[17] == 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_at_the_types_ends(dtype):
    """All logits at the lowest (or highest) value: an even row."""
    logits, experts = make(60, 24, 2, dtype)
    logits[19] = torch.finfo(logits.dtype).min
    logits[20] = torch.finfo(logits.dtype).max
    check(60, 24, 2, dtype, logits=logits, experts=experts)


@pytest.mark.parametrize("T", [100, 9000])
def test_nan_logits(T):
    logits, experts = make(T, 64, 2, "f32")
    logits[40, 3] = float("nan")
    loss, counts = ro.rowops_router_balance_loss(logits, experts, COEF)
    assert torch.isnan(loss).all()
    d = ro.rowops_router_balance_loss_backward(logits, counts, 2, torch.ones(1, device="cuda"), COEF)
    assert torch.isnan(d[40]).all() and torch.isfinite(d[:40]).all() and torch.isfinite(d[41:]).all()


@pytest.mark.parametrize("wide", [True, False])
def test_choices_outside_and_twice(wide):
    logits, experts = make(500, 16, 4, "f32", wide=wide)
    experts[::3, 0] = -1
    experts[::5, 1] = 16
    experts[1::7, 2] = torch.iinfo(experts.dtype).max
    experts[2::7, 2] = torch.iinfo(experts.dtype).min
    experts[3] = 2
    check(500, 16, 4, "f32", logits=logits, experts=experts)


def test_all_choose_one_expert():
    logits, experts = make(50000, 8, 2, "f32")
    check(50000, 8, 2, "f32", logits=logits, experts=torch.full_like(experts, 3))


@pytest.mark.parametrize("T", [64, 50000])
def test_in_place_given_workspace_and_repeatable(T):
    logits, experts, loss, counts, d = check(T, 64, 6, "bf16")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    a, c = ro.rowops_router_balance_loss(logits, experts, COEF, loss=torch.empty(1, device="cuda"),
                                         counts=torch.empty_like(counts), workspace=ws)
    assert torch.equal(a, loss) and torch.equal(c, counts)
    dl = torch.full((1,), 1.75, device="cuda")
    z = logits.clone()
    assert torch.equal(ro.rowops_router_balance_loss_backward(z, counts, 6, dl, COEF, None, z), d)


def test_no_rows_and_refusals():
    x = torch.empty(0, 8, device="cuda")
    loss, counts = ro.rowops_router_balance_loss(x, torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    assert float(loss) == 0 and torch.all(counts == 0)
    x, e = make(10, 8, 2, "f32")
    with pytest.raises(ValueError):
        ro.rowops_router_balance_loss(x, e[:5])
    with pytest.raises(ValueError):
        ro.rowops_router_balance_loss(x, e.t().contiguous().t())
    with pytest.raises(TypeError):
        ro.rowops_router_balance_loss(x, e.short())
    with pytest.raises(ValueError):
        ro.rowops_router_balance_loss(x, e, mask=torch.ones(9, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        ro.rowops_router_balance_loss_backward(x, torch.zeros(8, dtype=torch.int64, device="cuda"), 2,
                                               torch.ones(1, device="cuda"))
    big = torch.zeros(4, 1025, device="cuda")
    with pytest.raises(ro.RowopsError):
        ro.rowops_router_balance_loss(big, torch.zeros(4, 1, dtype=torch.int64, device="cuda"))
