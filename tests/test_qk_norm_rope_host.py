"""Refusals of the query/key norm + rotary calls (no GPU: the host-side checks
return before any launch)."""
import pytest

from megatron_tensor_transformer_logical_b200 import binding as L

P = [0x10000 * (i + 1) for i in range(16)]
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return L.load()


def fwd(lib, Q=P[0], ldq=1024, K=P[1], ldk=256, gq=P[2], gk=P[3], pos=P[4], fr=P[5], Qo=P[6],
        ldqo=1024, Ko=P[7], ldko=256, M=4, heads=8, kv=2, d=128, d_rot=128, norm=1, il=0,
        eps=1e-6, dt=L.TP_BF16):
    return lib.tp_qk_norm_rope_fwd(Q, ldq, K, ldk, gq, gk, pos, fr, Qo, ldqo, Ko, ldko, M, heads,
                                   kv, d, d_rot, norm, il, eps, dt, None)


def bwd(lib, Q=P[0], ldq=1024, K=P[1], ldk=256, gq=P[2], gk=P[3], pos=P[4], fr=P[5], dQo=P[6],
        lddqo=1024, dKo=P[7], lddko=256, dQ=P[8], lddq=1024, dK=P[9], lddk=256, dgq=P[10],
        dgk=P[11], M=4, heads=8, kv=2, d=128, d_rot=128, norm=1, il=0, eps=1e-6, dt=L.TP_BF16,
        ws=P[12], wsb=BIG):
    return lib.tp_qk_norm_rope_bwd(Q, ldq, K, ldk, gq, gk, pos, fr, dQo, lddqo, dKo, lddko, dQ,
                                   lddq, dK, lddk, dgq, dgk, M, heads, kv, d, d_rot, norm, il, eps,
                                   dt, ws, wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("bad,status", [
    (dict(Q=None), L.TP_ERR_NULL), (dict(K=None), L.TP_ERR_NULL), (dict(pos=None), L.TP_ERR_NULL),
    (dict(fr=None), L.TP_ERR_NULL), (dict(M=-1), L.TP_ERR_SHAPE), (dict(heads=0), L.TP_ERR_SHAPE),
    (dict(kv=-1), L.TP_ERR_SHAPE), (dict(d=0), L.TP_ERR_SHAPE), (dict(d=100), L.TP_ERR_ALIGN),
    (dict(d=264, d_rot=0), L.TP_ERR_UNSUPPORTED), (dict(d_rot=-16), L.TP_ERR_SHAPE),
    (dict(d_rot=144), L.TP_ERR_SHAPE), (dict(d_rot=24), L.TP_ERR_ALIGN),
    (dict(ldq=1016), L.TP_ERR_SHAPE), (dict(ldk=260), L.TP_ERR_ALIGN),
    (dict(ldq=1 << 32), L.TP_ERR_SHAPE), (dict(M=1 << 31), L.TP_ERR_SHAPE),
    (dict(heads=1 << 24, ldq=1 << 31), L.TP_ERR_SHAPE), (dict(Q=P[0] + 8), L.TP_ERR_ALIGN),
    (dict(gk=P[3] + 2), L.TP_ERR_ALIGN), (dict(fr=P[5] + 4), L.TP_ERR_ALIGN),
    (dict(pos=P[4] + 2), L.TP_ERR_ALIGN), (dict(dt=3), L.TP_ERR_DTYPE)])
def test_refusals(lib, call, bad, status):
    assert call(lib, **bad) == status
    assert lib.tp_last_error()


def test_refusals_of_outputs_and_workspace(lib):
    assert fwd(lib, Qo=None) == L.TP_ERR_NULL
    assert fwd(lib, Ko=None) == L.TP_ERR_NULL
    assert fwd(lib, ldko=248) == L.TP_ERR_SHAPE
    for bad in (dict(dQo=None), dict(dQ=None), dict(dKo=None), dict(dK=None)):
        assert bwd(lib, **bad) == L.TP_ERR_NULL
    assert bwd(lib, lddqo=8) == L.TP_ERR_SHAPE
    assert bwd(lib, lddk=257) == L.TP_ERR_ALIGN
    need = lib.tp_workspace_size(L.TP_OP_QK_NORM_ROPE_BWD, 4, 128, 0, 0, 1, L.TP_F16)
    assert need > 0
    assert bwd(lib, ws=None) == L.TP_ERR_WORKSPACE
    assert bwd(lib, wsb=need - 1) == L.TP_ERR_WORKSPACE
    assert lib.tp_workspace_size(L.TP_OP_QK_NORM_ROPE_BWD, 4, 512, 0, 0, 1, L.TP_BF16) == 0
    assert lib.tp_workspace_size(L.TP_OP_QK_NORM_ROPE_BWD, 4, 128, 0, 0, 1, 3) == 0


def test_no_tokens_is_a_no_op(lib):
    assert fwd(lib, M=0, Q=None, K=None, Qo=None, Ko=None, pos=None) == L.TP_OK


def test_the_older_calls_refuse_fp16(lib):
    assert lib.tp_linear_col(P[0], P[1], None, P[2], 64, 128, 256, 4, -1, L.TP_F16, L.TP_F16,
                             None) == L.TP_ERR_DTYPE
    assert lib.tp_layernorm_fwd(P[0], None, None, P[1], None, None, 4, 64, 1e-5, L.TP_F16,
                                None) == L.TP_ERR_DTYPE
    assert lib.tp_workspace_size(L.TP_OP_MLP_FWD, 64, 64, 64, 0, 1, L.TP_F16) == 0
