"""Refusals of the serving operators' C ABI: invalid arguments get the documented
status before any CUDA call (the pointers are fake)."""
import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
X, R, RO, Q, S, W = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000, 0x6000000
K, V, TABLE, LENGTHS, OUT, LSE, WS = 0x10000000, 0x20000000, 0x30000000, 0x31000000, 0x32000000, 0x33000000, 0x40000000


@pytest.fixture(scope="module")
def lib():
    from row_wise_reduction_gb300 import build
    from row_wise_reduction_gb300.rowops import library

    build.build()
    return library()


def test_rmsnorm_quant_refusals(lib):
    f = lib.rowops_rmsnorm_quant

    def args(x=X, r=R, q=Q, s=S, ro=RO, w=W, eps=1e-5, M=4, N=64, ld=64, ldq=64, group=32, dt=F32):
        return (x, r, q, s, ro, w, eps, M, N, ld, ldq, group, dt, None)

    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(ro=None), dict(r=None), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(M=-1), dict(N=0), dict(ld=63), dict(ldq=63),
                dict(group=-32), dict(group=31), dict(group=48), dict(dt=2), dict(x=X + 2), dict(r=R + 1),
                dict(ro=RO + 2), dict(w=W + 2), dict(s=S + 2), dict(ro=X + 16), dict(ro=R + 16),
                dict(q=X), dict(q=X + 1000), dict(q=R), dict(q=RO + 4), dict(q=W), dict(q=S),
                dict(s=X), dict(s=R), dict(s=RO), dict(s=W + 4), dict(s=Q + 4), dict(w=RO)):
        assert f(*args(**bad)) == INVALID, bad
    for bad in (dict(N=1 << 31, ld=1 << 31, ldq=1 << 31), dict(M=1 << 40, ld=1 << 40), dict(M=1 << 40, ldq=1 << 40, r=None, ro=None)):
        assert f(*args(**bad)) == UNSUPPORTED, bad
    assert f(*args(M=0, x=None, r=None, q=None, s=None, ro=None)) == OK
    assert f(*args(M=0, group=16)) == INVALID  # checked all the same


def test_paged_attention_refusals(lib):
    f, g = lib.rowops_paged_attention, lib.rowops_paged_attention_workspace_bytes
    assert g(1, 8, 2, 64, 16, 5, 0, BF16) == 0  # one kernel
    need = g(300, 8, 2, 64, 16, 500, 0, BF16)
    assert need > 0 and g(300, 8, 2, 64, 16, 500, 10**9, BF16) == need
    for window in (8000, 2**63 - 15, 2**63 - 1):  # as none
        assert g(4, 8, 2, 64, 16, 500, window, BF16) == g(4, 8, 2, 64, 16, 500, 0, BF16) > 0, window
    for bad in ((0, 8, 2, 64, 16, 500, 0, BF16), (300, 7, 2, 64, 16, 500, 0, BF16), (300, 8, 0, 64, 16, 500, 0, BF16),
                (300, 8, 2, 257, 16, 500, 0, BF16), (300, 8, 2, 0, 16, 500, 0, BF16), (300, 8, 2, 64, 16, 500, 0, 7),
                (1 << 31, 8, 2, 64, 16, 500, 0, BF16), ((1 << 24) + 1, 2, 2, 64, 16, 500, 0, BF16), (300, 8, 2, 64, 0, 500, 0, BF16), (300, 8, 2, 64, 16, -1, 0, BF16),
                (300, 8, 2, 64, 16, 500, -1, BF16), (300, 8, 2, 64, 16, 1 << 30, 0, BF16)):
        assert g(*bad) == 0, bad

    def args(q=X, k=K, v=V, table=TABLE, lengths=LENGTHS, out=OUT, lse=LSE, scale=0.125, window=0, B=300, H=8, KV=2, D=64,
             ldq=512, ldo=512, pages=10, page=16, ps=2048, ss=128, hs=64, width=500, ldt=500, dt=BF16, ws=WS, nb=None):
        return (q, k, v, table, lengths, out, lse, scale, window, B, H, KV, D, ldq, ldo, pages, page, ps, ss, hs, width,
                ldt, dt, ws, need if nb is None else nb, None)

    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lengths=None), dict(out=None),
                dict(scale=float("nan")), dict(scale=float("inf")),
                dict(scale=-3e38), dict(window=-1), dict(B=-1), dict(H=0), dict(KV=0),
                dict(KV=3), dict(D=0), dict(ldq=511), dict(ldo=511), dict(pages=-1), dict(page=0), dict(ps=-1),
                dict(ss=-1), dict(hs=-1), dict(width=-1), dict(ldt=499), dict(dt=2), dict(q=X + 1), dict(k=K + 1),
                dict(v=V + 1), dict(out=OUT + 1), dict(table=TABLE + 2), dict(lengths=LENGTHS + 2), dict(lse=LSE + 2),
                dict(out=X), dict(out=X + 64), dict(out=K + 64), dict(out=V), dict(out=TABLE), dict(out=LENGTHS),
                dict(lse=X), dict(lse=K), dict(lse=V + 4), dict(lse=TABLE), dict(lse=LENGTHS), dict(lse=OUT)):
        assert f(*args(**bad)) == INVALID, bad
    for bad in (dict(D=257, ldq=4096, ldo=4096), dict(B=1 << 31), dict(B=(1 << 24) + 1, H=2), dict(page=1 << 31), dict(pages=1 << 32),
                dict(width=1 << 31, ldt=1 << 31), dict(ps=1 << 62), dict(ss=1 << 62), dict(hs=1 << 62),
                dict(ldq=1 << 62), dict(ldt=1 << 62)):
        assert f(*args(**bad)) == UNSUPPORTED, bad
    assert f(*args(B=0, q=None, k=None, v=None, table=None, lengths=None, out=None, ws=None)) == OK
    for bad in (dict(ws=None), dict(ws=WS + 128), dict(nb=need - 1)):
        assert f(*args(**bad)) == WORKSPACE, bad
    for bad in (dict(ws=X), dict(ws=K), dict(ws=V), dict(ws=TABLE), dict(ws=LENGTHS), dict(ws=OUT), dict(ws=LSE)):
        assert f(*args(**bad)) == INVALID, bad


def test_sample_refusals(lib):
    f = lib.rowops_sample
    U, T, TK, TP, MP, TOKEN, LP = (0x7000000 + 0x100000 * i for i in range(7))

    def args(x=X, u=U, t=T, ta=1.0, k=TK, ka=0, p=TP, pa=1.0, m=MP, ma=0.0, token=TOKEN, lp=LP, M=4, N=64, ld=64, dt=F32):
        return (x, u, t, ta, k, ka, p, pa, m, ma, token, lp, M, N, ld, dt, None)

    nan = float("nan")
    for bad in (dict(x=None), dict(u=None), dict(token=None), dict(ta=-1.0), dict(ta=nan), dict(ka=-1), dict(pa=-0.1),
                dict(pa=nan), dict(ma=-0.1), dict(ma=1.5), dict(ma=nan), dict(M=-1), dict(N=0), dict(ld=63), dict(dt=9),
                dict(x=X + 2), dict(u=U + 2), dict(t=T + 1), dict(k=TK + 2), dict(p=TP + 2), dict(m=MP + 2),
                dict(token=TOKEN + 4), dict(lp=LP + 2), dict(token=X), dict(token=U), dict(token=T), dict(token=TK),
                dict(token=TP), dict(token=MP), dict(token=LP), dict(lp=X + 64), dict(lp=U), dict(lp=T),
                dict(lp=TK + 4), dict(lp=TP), dict(lp=MP)):
        assert f(*args(**bad)) == INVALID, bad
    for bad in (dict(N=327681, ld=327681), dict(M=(1 << 27) + 1)):
        assert f(*args(**bad)) == UNSUPPORTED, bad
    assert f(*args(M=0, x=None, u=None, token=None)) == OK
