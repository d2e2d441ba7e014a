"""Refusals of the training operators' C ABI: invalid arguments get the
documented status before any CUDA call (the pointers are fake)."""
import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
X, Y, DY, DX = 0x1000000, 0x2000000, 0x3000000, 0x4000000
W, BI, STATS, DW, DB, WS = 0x5000000, 0x5100000, 0x5200000, 0x5300000, 0x5400000, 0x6000000


@pytest.fixture(scope="module")
def lib():
    from row_wise_reduction_gb300 import build
    from row_wise_reduction_gb300.rowops import library

    build.build()
    return library()


def test_groupnorm_refusals(lib, monkeypatch):
    q = lib.rowops_groupnorm_act_workspace_bytes
    assert q(2, 16, 64, 8, F32) == 0  # one kernel: no workspace
    monkeypatch.setenv("ROWOPS_GROUPNORM", "stream")
    f, q = lib.rowops_groupnorm_act, lib.rowops_groupnorm_act_workspace_bytes
    need = q(2, 16, 64, 8, F32)
    assert need > 0 and q(0, 16, 64, 8, F32) == 0 and q(2, 16, 64, 7, F32) == 0 and q(2, 16, 64, 8, 5) == 0

    def args(x=X, y=Y, w=W, b=BI, eps=1e-5, B=2, S=16, C=64, G=8, ld=64, act=1, stats=STATS, dt=F32, ws=WS, nb=None):
        return (x, y, w, b, eps, B, S, C, G, ld, act, stats, dt, ws, need if nb is None else nb, None)

    for bad in (dict(x=None), dict(y=None), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(B=-1), dict(S=-1), dict(C=0), dict(G=0), dict(G=7), dict(ld=63), dict(act=4), dict(act=-1),
                dict(dt=2), dict(x=X + 2), dict(w=W + 2), dict(b=BI + 1), dict(stats=STATS + 4),
                dict(y=X + 16),                         # y partly overlaps x
                dict(w=Y + 64), dict(b=Y + 64),         # written while read
                dict(stats=X + 64), dict(stats=Y + 64), dict(stats=W), dict(stats=BI + 8),
                dict(ws=X), dict(ws=Y), dict(ws=W), dict(ws=STATS)):
        assert f(*args(**bad)) == INVALID, bad
    for bad in (dict(C=8200, ld=8200, G=8), dict(B=1 << 31), dict(B=1 << 30, S=1 << 40)):
        assert f(*args(**bad)) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=WS + 128), dict(nb=need - 1)):
        assert f(*args(**bad)) == WORKSPACE, bad
    for none in (dict(B=0), dict(S=0)):
        assert f(*args(x=None, y=None, ws=None, nb=0, **none)) == OK


def test_groupnorm_backward_refusals(lib, monkeypatch):
    q = lib.rowops_groupnorm_act_backward_workspace_bytes
    assert q(3, 16, 64, 8, F32) >= 3 * 64 * 8  # one kernel: the samples' channel sums
    monkeypatch.setenv("ROWOPS_GROUPNORM", "stream")
    f, q = lib.rowops_groupnorm_act_backward, lib.rowops_groupnorm_act_backward_workspace_bytes
    need = q(2, 16, 64, 8, BF16)
    assert need > 0 and q(2, -1, 64, 8, BF16) == 0

    def args(x=X, dy=DY, w=W, b=BI, stats=STATS, dx=DX, dw=DW, db=DB, B=2, S=16, C=64, G=8, ld=64, act=1, dt=BF16,
             ws=WS, nb=None):
        return (x, dy, w, b, stats, dx, dw, db, B, S, C, G, ld, act, dt, ws, need if nb is None else nb, None)

    for bad in (dict(x=None), dict(dy=None), dict(dx=None), dict(stats=None), dict(dw=None), dict(db=None),
                dict(dx=X), dict(dx=DY), dict(dx=X + 32), dict(db=DW), dict(db=DW + 64), dict(dw=DX), dict(db=DX + 4),
                dict(dw=X), dict(db=DY), dict(dw=W), dict(db=STATS), dict(stats=DX + 8), dict(w=DX), dict(b=DX),
                dict(dw=DW + 2), dict(stats=STATS + 4), dict(w=W + 1), dict(b=BI + 1), dict(G=9), dict(act=7),
                dict(ld=60), dict(dt=3), dict(ws=DX), dict(ws=X), dict(ws=DY), dict(ws=STATS), dict(ws=DW),
                dict(ws=DB), dict(ws=W)):
        assert f(*args(**bad)) == INVALID, bad
    assert f(*args(C=16384, G=8, ld=16384)) == UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=WS + 64), dict(nb=need - 1)):
        assert f(*args(**bad)) == WORKSPACE, bad


def test_dropout_refusals(lib):
    f, g = lib.rowops_bias_dropout_residual, lib.rowops_bias_dropout_residual_backward
    q = lib.rowops_bias_dropout_residual_backward_workspace_bytes
    need = q(4, 64, F32)
    assert need == 4 * 64 * 4 and q(1 << 20, 8192, BF16) == 512 * 8192 * 4
    assert q(-1, 8, F32) == 0 and q(4, 0, F32) == 0 and q(4, 8, 9) == 0

    def fwd(x=X, r=DY, b=BI, y=Y, p=0.1, off=None, M=4, N=64, ld=64, dt=F32):
        return (x, r, b, y, p, 1, 2, off, M, N, ld, dt, None)

    def bwd(dy=DY, dx=DX, db=DB, p=0.1, off=None, M=4, N=64, ld=64, dt=F32, ws=WS, nb=None):
        return (dy, dx, db, p, 1, 2, off, M, N, ld, dt, ws, need if nb is None else nb, None)

    for bad in (dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(x=None), dict(y=None), dict(y=X + 16),
                dict(y=DY + 16), dict(b=Y + 4), dict(b=BI + 2), dict(off=Y + 8), dict(off=STATS + 4), dict(ld=63),
                dict(dt=2), dict(N=0), dict(M=-1), dict(r=DY + 2)):
        assert f(*fwd(**bad)) == INVALID, bad
    assert f(*fwd(M=(1 << 32) + 1)) in (INVALID, UNSUPPORTED)  # such a span also overlaps the other fake pointers
    assert f(X, None, None, X, 0.1, 1, 2, None, (1 << 32) + 1, 1, 1, F32, None) == UNSUPPORTED
    assert f(*fwd(N=1 << 31, ld=1 << 31)) == UNSUPPORTED
    assert f(*fwd(M=0)) == OK
    for bad in (dict(p=2.0), dict(dy=None), dict(dx=DY + 16), dict(db=DX), dict(db=DY), dict(db=DB + 2),
                dict(off=DX), dict(off=DB), dict(ws=DY), dict(ws=DX), dict(ws=DB), dict(ld=1)):
        assert g(*bwd(**bad)) == INVALID, bad
    for bad in (dict(ws=None), dict(ws=WS + 16), dict(nb=need - 1)):
        assert g(*bwd(**bad)) == WORKSPACE, bad
    assert g(*bwd(M=0, db=None, ws=None, nb=0)) == OK


def test_router_refusals(lib):
    f, g = lib.rowops_router_balance_loss, lib.rowops_router_balance_loss_backward
    q = lib.rowops_router_balance_loss_workspace_bytes
    assert q(64, 8, F32) == 0 and q(-1, 8, F32) == 0 and q(64, 2000, F32) == 0
    need = q(100000, 64, F32)
    assert need == 128 * (2 * 64 + 1) * 4
    LOSS, CNT, EXP, MASK = STATS, DW, DY, W

    def fwd(x=X, e=EXP, ib=8, m=MASK, coef=0.1, loss=LOSS, c=CNT, T=16, E=8, K=2, ld=8, dt=F32, ws=None, nb=0):
        return (x, e, ib, m, coef, loss, c, T, E, K, ld, dt, ws, nb, None)

    def bwd(x=X, c=CNT, dl=LOSS, m=MASK, coef=0.1, dx=DX, T=16, E=8, K=2, ld=8, dt=F32):
        return (x, c, dl, m, coef, dx, T, E, K, ld, dt, None)

    for bad in (dict(x=None), dict(e=None), dict(ib=2), dict(K=0), dict(coef=float("nan")), dict(coef=float("inf")),
                dict(loss=None), dict(c=None), dict(loss=LOSS + 2), dict(c=CNT + 4), dict(e=EXP + 4), dict(ld=7),
                dict(dt=4), dict(loss=CNT + 8), dict(loss=X), dict(c=X + 8), dict(c=EXP), dict(loss=MASK)):
        assert f(*fwd(**bad)) == INVALID, bad
    big = dict(T=100000, E=64, ld=64, x=0x10000000, e=0x20000000, m=0x30000000)
    for bad in (dict(ws=None), dict(ws=WS + 8, nb=need), dict(ws=WS, nb=need - 1)):
        assert f(*fwd(**big, **bad)) == WORKSPACE, bad
    for bad in (dict(ws=0x10000000, nb=need), dict(ws=0x20000000, nb=need), dict(ws=0x30000000, nb=need),
                dict(ws=CNT, nb=need)):
        assert f(*fwd(**big, **bad)) == INVALID, bad
    assert f(*fwd(E=1025, ld=1025)) == UNSUPPORTED
    assert f(*fwd(T=1 << 30, K=2, m=None)) == UNSUPPORTED
    for bad in (dict(x=None), dict(c=None), dict(dl=None), dict(dx=None), dict(K=0), dict(coef=float("inf")),
                dict(dx=X + 16), dict(dx=CNT), dict(dx=LOSS), dict(dx=MASK), dict(c=CNT + 4), dict(dl=LOSS + 1)):
        assert g(*bwd(**bad)) == INVALID, bad
    assert g(*bwd(E=1025, ld=1025)) == UNSUPPORTED
    assert g(*bwd(T=0)) == OK


def test_binding_refuses_host_tensors():
    import torch

    import row_wise_reduction_gb300 as ro

    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ro.rowops_groupnorm_act(x.reshape(1, 4, 8), 2)
    with pytest.raises(ValueError):
        ro.rowops_bias_dropout_residual(x)
    with pytest.raises(ValueError):
        ro.rowops_bias_dropout_residual_backward(x)
    with pytest.raises(ValueError):
        ro.rowops_router_balance_loss(x, torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        ro.rowops_router_balance_loss_backward(x, torch.zeros(9, dtype=torch.int64), 2, torch.ones(1))
