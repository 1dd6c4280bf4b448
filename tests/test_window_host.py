"""Refusals and workspace sizes of the window attention calls (no GPU: the
host-side checks return before any launch)."""
import pytest

from megatron_tensor_transformer_logical_b200 import binding as L

P = [0x10000 * (i + 1) for i in range(16)]
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return L.load()


def fwd(lib, Q=P[0], ldq=1024, K=P[1], ldk=256, V=P[2], ldv=256, O=P[3], ldo=1024, LSE=P[4], b=2,
        sq=64, sk=64, heads=8, kv=2, d=128, W=32, S=4, scale=0.0, dt=L.TP_BF16):
    return lib.tp_window_attn_fwd(Q, ldq, K, ldk, V, ldv, O, ldo, LSE, b, sq, sk, heads, kv, d, W,
                                  S, scale, dt, None)


def bwd(lib, Q=P[0], ldq=1024, K=P[1], ldk=256, V=P[2], ldv=256, O=P[3], ldo=1024, LSE=P[4],
        dO=P[5], lddo=1024, dQ=P[6], lddq=1024, dK=P[7], lddk=256, dV=P[8], lddv=256, b=2, sq=64,
        sk=64, heads=8, kv=2, d=128, W=32, S=4, scale=0.0, dt=L.TP_BF16, ws=P[9], wsb=BIG):
    return lib.tp_window_attn_bwd(Q, ldq, K, ldk, V, ldv, O, ldo, LSE, dO, lddo, dQ, lddq, dK,
                                  lddk, dV, lddv, b, sq, sk, heads, kv, d, W, S, scale, dt, ws,
                                  wsb, None)


def dec(lib, Q=P[0], ldq=1024, K=P[1], ldk=256, bk=1 << 16, V=P[2], ldv=256, bv=1 << 16, lens=P[3],
        O=P[4], ldo=1024, LSE=P[5], b=2, sk=64, heads=8, kv=2, d=128, W=32, S=4, scale=0.0,
        dt=L.TP_BF16, ws=P[6], wsb=BIG):
    return lib.tp_window_attn_decode(Q, ldq, K, ldk, bk, V, ldv, bv, lens, O, ldo, LSE, b, sk,
                                     heads, kv, d, W, S, scale, dt, ws, wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd, dec])
@pytest.mark.parametrize("bad,status", [
    (dict(Q=None), L.TP_ERR_NULL), (dict(K=None), L.TP_ERR_NULL), (dict(V=None), L.TP_ERR_NULL),
    (dict(O=None), L.TP_ERR_NULL), (dict(b=0), L.TP_ERR_SHAPE), (dict(sk=0), L.TP_ERR_SHAPE),
    (dict(heads=0), L.TP_ERR_SHAPE), (dict(kv=0), L.TP_ERR_SHAPE), (dict(kv=3), L.TP_ERR_SHAPE),
    (dict(d=96), L.TP_ERR_UNSUPPORTED), (dict(W=0), L.TP_ERR_SHAPE), (dict(S=-1), L.TP_ERR_SHAPE),
    (dict(scale=-1.0), L.TP_ERR_SHAPE), (dict(scale=float("nan")), L.TP_ERR_SHAPE),
    (dict(scale=float("inf")), L.TP_ERR_SHAPE), (dict(ldq=1016), L.TP_ERR_SHAPE),
    (dict(ldk=257), L.TP_ERR_ALIGN), (dict(ldv=128), L.TP_ERR_SHAPE),
    (dict(ldo=1 << 33), L.TP_ERR_SHAPE), (dict(V=P[2] + 8), L.TP_ERR_ALIGN),
    (dict(dt=L.TP_F32), L.TP_ERR_DTYPE), (dict(dt=5), L.TP_ERR_DTYPE),
    (dict(sk=1 << 32), L.TP_ERR_SHAPE), (dict(b=1 << 30), L.TP_ERR_SHAPE)])
def test_refusals(lib, call, bad, status):
    assert call(lib, **bad) == status
    assert lib.tp_last_error()


def test_refusals_of_the_single_calls(lib):
    assert fwd(lib, LSE=None) == L.TP_ERR_NULL
    assert fwd(lib, sq=0) == L.TP_ERR_SHAPE
    assert fwd(lib, sq=1 << 31) == L.TP_ERR_SHAPE
    for bad in (dict(dO=None), dict(dQ=None), dict(dK=None), dict(dV=None)):
        assert bwd(lib, **bad) == L.TP_ERR_NULL
    assert bwd(lib, lddo=1000) == L.TP_ERR_SHAPE
    assert bwd(lib, lddv=252) == L.TP_ERR_SHAPE
    assert bwd(lib, dK=P[7] + 2) == L.TP_ERR_ALIGN
    need = lib.tp_window_attn_workspace_size(2, 64, 64, 8, 2, 128, 32, 4)
    assert need >= 2 * 2 * 8 * 64 * 4
    assert bwd(lib, ws=None) == L.TP_ERR_WORKSPACE
    assert bwd(lib, wsb=need - 1) == L.TP_ERR_WORKSPACE
    assert dec(lib, lens=None) == L.TP_ERR_NULL
    assert dec(lib, bk=12) == L.TP_ERR_ALIGN
    assert dec(lib, bv=-8) == L.TP_ERR_SHAPE
    assert dec(lib, ws=None) == L.TP_ERR_WORKSPACE
    need = lib.tp_window_decode_workspace_size(2, 1 << 17, 8, 2, 128, 1 << 17, 0)
    assert dec(lib, sk=1 << 17, W=1 << 17, wsb=need - 1) == L.TP_ERR_WORKSPACE


def test_workspace_sizes(lib):
    ws, wd = lib.tp_window_attn_workspace_size, lib.tp_window_decode_workspace_size
    assert ws(2, 64, 64, 8, 3, 128, 32, 4) == 0 and ws(2, 0, 64, 8, 2, 128, 32, 4) == 0
    assert wd(0, 64, 8, 2, 128, 32, 4) == 0 and wd(2, 64, 8, 2, 80, 32, 4) == 0
    # The partials stay bounded.  A slice takes C >= blocks / (2 SMs) of all
    # blocks; tiles are cut only if the longest, m, exceeds C, and with tiles
    # between 0 and m blocks long (m / 2 on average) that means fewer than 4 SMs
    # tiles of m / C + 1 slices each: below 8 slices per SM.
    for b, s, h, kv, w, sk in ((1, 1 << 20, 64, 1, 1 << 20, 0), (1, 1 << 17, 64, 8, 1024, 4),
                               (64, 4096, 32, 8, 512, 128), (1, 8192, 8, 8, 8192, 0)):
        stats = 2 * (b * h * s + 64) * 4 + 512
        assert ws(b, s, s, h, kv, 128, w, sk) - stats <= 8 * 160 * 2 * 128 * 128 * 4


@pytest.mark.parametrize("heads,kv,cap,window,sinks", [
    (32, 8, 8192, 4096, 4), (32, 4, 131072, 131072, 0), (40, 1, 3000, 700, 3), (8, 8, 300, 300, 0)])
def test_a_decode_workspace_serves_smaller_batches(lib, heads, kv, cap, window, sinks):
    size = lambda b: lib.tp_window_decode_workspace_size(b, cap, heads, kv, 128, window, sinks)
    sizes = [size(b) for b in range(1, 400)]
    assert sizes == sorted(sizes)
    # what the launch lays out: a slice per 256 keys at most, enough of them for
    # two blocks per SM (148 of them; without a GPU the library plans for as many)
    group = heads // kv
    for b, have in zip(range(1, 400), sizes):
        items, keys = b * kv * -(-group // 16), min(cap, window + sinks)
        splits = max(1, min(-(-2 * 148 // items), -(-keys // 256), 255))
        rows = items * splits * min(group, 16) if splits > 1 else 0
        assert have >= -(-rows * 8 // 256) * 256 + rows * 128 * 4
