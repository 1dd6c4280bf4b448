"""Refusals of the gated feed-forward calls (no GPU: the host-side checks
return before any launch)."""
import pytest

from megatron_tensor_transformer_logical_b200 import binding as L

P = [0x10000 * (i + 1) for i in range(16)]
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return L.load()


def fwd(lib, X=P[0], Wgu=P[1], bgu=P[2], Wd=P[3], bd=P[4], Z=P[5], GU=P[6], M=100, h=128, f=512,
        t=4, act=L.TP_ACT_SILU, dt=L.TP_BF16, ws=P[7], wsb=BIG):
    return lib.tp_glu_fwd(X, Wgu, bgu, Wd, bd, Z, GU, M, h, f, t, act, dt, ws, wsb, None)


def bwd(lib, X=P[0], Wgu=P[1], bgu=P[2], Wd=P[3], GU=P[6], dZ=P[5], dX=P[8], dWgu=P[9], dbgu=P[10],
        dWd=P[11], dbd=P[12], M=100, h=128, f=512, t=4, act=L.TP_ACT_GELU, dt=L.TP_BF16, ws=P[7],
        wsb=BIG):
    return lib.tp_glu_bwd(X, Wgu, bgu, Wd, GU, dZ, dX, dWgu, dbgu, dWd, dbd, M, h, f, t, act, dt,
                          ws, wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("bad,status", [
    (dict(X=None), L.TP_ERR_NULL), (dict(Wgu=None), L.TP_ERR_NULL), (dict(Wd=None), L.TP_ERR_NULL),
    (dict(M=0), L.TP_ERR_SHAPE), (dict(h=-8), L.TP_ERR_SHAPE), (dict(f=0), L.TP_ERR_SHAPE),
    (dict(f=520, t=3), L.TP_ERR_SHAPE), (dict(t=0), L.TP_ERR_SHAPE), (dict(t=65), L.TP_ERR_SHAPE),
    (dict(h=132), L.TP_ERR_ALIGN), (dict(f=516), L.TP_ERR_ALIGN), (dict(f=1 << 30), L.TP_ERR_SHAPE),
    (dict(M=1 << 31), L.TP_ERR_SHAPE), (dict(f=1 << 62, t=1), L.TP_ERR_SHAPE),
    (dict(X=P[0] + 8), L.TP_ERR_ALIGN), (dict(bgu=P[2] + 2), L.TP_ERR_ALIGN),
    (dict(GU=P[6] + 4), L.TP_ERR_ALIGN), (dict(act=2), L.TP_ERR_UNSUPPORTED),
    (dict(dt=L.TP_F32), L.TP_ERR_UNSUPPORTED), (dict(dt=L.TP_F16), L.TP_ERR_DTYPE),
    (dict(ws=None), L.TP_ERR_WORKSPACE), (dict(wsb=1024), L.TP_ERR_WORKSPACE)])
def test_refusals(lib, call, bad, status):
    assert call(lib, **bad) == status
    assert lib.tp_last_error()


def test_refusals_of_outputs(lib):
    assert fwd(lib, Z=None) == L.TP_ERR_NULL
    for bad in (dict(dZ=None), dict(dX=None), dict(dWgu=None), dict(dWd=None)):
        assert bwd(lib, **bad) == L.TP_ERR_NULL
    assert bwd(lib, dbd=P[12] + 2) == L.TP_ERR_ALIGN


def test_workspace_sizes(lib):
    ws = lambda op, M, h, f, dt=L.TP_BF16: lib.tp_workspace_size(op, M, h, f, 0, 1, dt)
    assert ws(L.TP_OP_GLU_FWD, 100, 128, 512) >= 100 * 512 * 2
    assert ws(L.TP_OP_GLU_BWD, 100, 128, 512) >= 5 * 100 * 512 * 2
    assert ws(L.TP_OP_GLU_FWD, 100, 128, 0) == 0
    assert ws(L.TP_OP_GLU_FWD, 100, 128, 512, L.TP_F32) == 0
    assert ws(L.TP_OP_GLU_BWD, 100, 128, 1 << 40) == 0


def test_a_forward_workspace_serves_fewer_tokens(lib):
    for f in (8, 2816, 14336):
        sizes = [lib.tp_workspace_size(L.TP_OP_GLU_FWD, M, 1024, f, 0, 1, L.TP_BF16)
                 for M in range(1, 70)]
        assert sizes == sorted(sizes)
