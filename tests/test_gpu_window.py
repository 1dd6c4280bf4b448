"""Window attention with sinks against fp64 (GPU): forward, backward, and the
single-token form over a cache.

Tolerances follow the roundings.  With hs half a step of the type (2^-8 bf16,
2^-11 fp16): P is rounded to the type (hs relative, the sum of P is not), so
|dO| <= hs (P |V|) + hs |O|; D = rowsum(dO * O) inherits the error eO of the
rounded O, eD = |dO| . eO; dS = P (dP - D) is rounded too, so |d dS| <=
hs |dS| + P eD, and dQ, dK, dV follow by linearity, each rounded once more.
The fp32 parts (products, exponentials to 2^-22, P recomputed from LSE) stay
below 2^-13 of the same magnitudes, taken with dP and D apart.  The type's
smallest step bounds what underflows.
"""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
F32 = 2.0 ** -13


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def visible(sq, sk, window, sinks):
    p = torch.arange(sq, device="cuda")[:, None] + sk - sq
    c = torch.arange(sk, device="cuda")[None, :]
    return (c <= p) & ((p - c < window) | (c < sinks))


def reference(Q, K, V, b, heads, kv, window, sinks, scale, dO=None):
    """Results and tolerances, fp64, dense."""
    dt, hs = Q.dtype, half_step(Q.dtype)
    tiny = 2.0 ** -24 if dt == FP else 0.0
    sq, sk, d = Q.shape[0] // b, K.shape[0] // b, Q.shape[1] // heads
    G = heads // kv
    seen = visible(sq, sk, window, sinks)
    z = lambda n, h: torch.zeros(b, n, h, d, dtype=torch.float64, device="cuda")
    o = {"O": z(sq, heads), "dQ": z(sq, heads), "dK": z(sk, kv), "dV": z(sk, kv)}
    t = {k: torch.zeros_like(v) for k, v in o.items()}
    lse = torch.zeros(b, heads, sq, dtype=torch.float64, device="cuda")
    tl = torch.zeros_like(lse)
    q4, k4, v4 = Q.reshape(b, sq, heads, d), K.reshape(b, sk, kv, d), V.reshape(b, sk, kv, d)
    for i in range(b):
        for h in range(heads):
            q, k, v = q4[i, :, h].double(), k4[i, :, h // G].double(), v4[i, :, h // G].double()
            s = (q @ k.t() * scale).masked_fill(~seen, float("-inf"))
            l = torch.logsumexp(s, 1)
            P = torch.where(seen, torch.exp(s - l[:, None]), torch.zeros_like(s))
            O = P @ v
            # Below 2^-14 an fp16 P is off by up to 2^-25, half its smallest step, not
            # by hs of itself; the row sum it is divided by is at least 1, since the
            # maximum in use is that of keys the row has seen.  So the seen keys add
            # 2^-25 |V| each (tiny / 2), which shows where sharp rows make O small.
            eO = hs * (P @ v.abs()) + hs * O.abs() + F32 * (P @ v.abs()) + tiny
            eO = eO + tiny / 2 * (seen.double() @ v.abs())
            o["O"][i, :, h], t["O"][i, :, h] = O, eO
            lse[i, h] = l
            tl[i, h] = 2.0 ** -20 * (1 + (q.abs() @ k.abs().t()).amax(1) * scale)
            if dO is None:
                continue
            g = dO.reshape(b, sq, heads, d)[i, :, h].double()
            dP, D = g @ v.t(), (g * O).sum(1, keepdim=True)
            dS = P * (dP - D)
            mag = P * (g.abs() @ v.abs().t() + (g.abs() * (P @ v.abs())).sum(1, keepdim=True))
            eS = hs * dS.abs() + P * (g.abs() * eO).sum(1, keepdim=True) + F32 * mag + tiny
            o["dQ"][i, :, h] = scale * dS @ k
            t["dQ"][i, :, h] = scale * eS @ k.abs() + hs * (scale * dS @ k).abs() + tiny
            o["dK"][i, :, h // G] += scale * dS.t() @ q
            t["dK"][i, :, h // G] += scale * eS.t() @ q.abs()
            o["dV"][i, :, h // G] += P.t() @ g
            t["dV"][i, :, h // G] += (hs + F32) * (P.t() @ g.abs()) + tiny * g.abs().sum(0)
    for n in ("dK", "dV"):
        t[n] += hs * o[n].abs() + tiny
    for dct in (o, t):
        for n in dct:
            dct[n] = dct[n].reshape(-1, dct[n].shape[2] * d)
    o["LSE"], t["LSE"] = lse, tl
    return o, t


def close(got, ref, tol, what):
    got = got.double()
    same = got == ref  # infinities of rows that see nothing
    err = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    bad = (err - tol).max().item()
    assert bad <= 0, f"{what}: {bad:.3e} over; worst error {err.max().item():.3e}"


def rn(g, *s, dt=BF, std=1.0):
    return (torch.randn(*s, generator=g, device="cuda") * std).to(dt)


def make(b, sq, sk, heads, kv, d, dt, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = rn(g, b * sk, (heads + 2 * kv) * d, dt=dt)
    K, V = qkv[:, heads * d:(heads + kv) * d], qkv[:, (heads + kv) * d:]
    Q = (qkv if sq == sk else rn(g, b * sq, (heads + kv) * d, dt=dt))[:, :heads * d]
    if std != 1.0:
        Q.mul_(std)
    return Q, K, V, rn(g, b * sq, heads * d, dt=dt)


def run(Q, K, V, dO, b, heads, kv, window, sinks, scale=0.0, ws=None):
    nan = lambda x: torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
    sq, sk, d = Q.shape[0] // b, K.shape[0] // b, Q.shape[1] // heads
    O, LSE = nan(Q), torch.full((b, heads, sq), float("nan"), device="cuda")
    L.tp_window_attn_fwd(Q, K, V, O, LSE, b, heads, kv, window, sinks, scale)
    if dO is None:
        return {"O": O, "LSE": LSE}
    if ws is None:
        ws = L.window_attn_workspace(b, sq, sk, heads, kv, d, window, sinks)
        ws.fill_(0xff)  # NaN wherever the call does not write before it reads
    dQ, dK, dV = nan(Q), nan(K), nan(V)
    L.tp_window_attn_bwd(Q, K, V, O, LSE, dO, dQ, dK, dV, b, heads, kv, window, sinks, ws, scale)
    return {"O": O, "LSE": LSE, "dQ": dQ, "dK": dK, "dV": dV}


CASES = [  # b, sq, sk, heads, kv_heads, d, window, sinks, dtype
    (1, 1, 1, 1, 1, 128, 1, 0, BF),
    (2, 3, 3, 2, 1, 64, 2, 1, FP),
    (1, 127, 127, 2, 2, 128, 16, 0, BF),
    (2, 128, 128, 4, 2, 64, 128, 4, BF),
    (1, 129, 129, 3, 1, 128, 5, 2, FP),
    (3, 257, 257, 2, 1, 128, 1, 0, BF),
    (1, 385, 385, 4, 4, 64, 64, 300, BF),
    (2, 700, 700, 6, 2, 128, 129, 130, BF),
    (1, 1000, 1000, 8, 1, 128, 100, 4, BF),     # one key head: sliced key tiles
    (1, 1900, 1900, 4, 1, 64, 1900, 0, FP),     # full causal, sliced
    (2, 515, 515, 2, 2, 128, 1 << 40, 7, BF),   # window past the end
    (1, 1, 300, 4, 2, 128, 64, 3, BF),          # one query at the end of its keys
    (2, 70, 700, 4, 1, 64, 90, 1, BF),          # queries at the end of longer keys
    (1, 300, 1300, 2, 2, 128, 256, 0, FP),
    (2, 300, 170, 2, 1, 128, 40, 2, BF),        # first 130 queries see nothing
    (1, 600, 130, 2, 2, 64, 500, 0, BF),        # a whole tile sees nothing
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%dq%dk%dh%d_%dd%dw%ds%d" % c[:8])
def test_forward_and_backward(case):
    b, sq, sk, heads, kv, d, window, sinks, dt = case
    Q, K, V, dO = make(b, sq, sk, heads, kv, d, dt)
    got = run(Q, K, V, dO, b, heads, kv, window, sinks)
    ref, tol = reference(Q, K, V, b, heads, kv, window, sinks, d ** -0.5, dO)
    for n in ref:
        close(got[n], ref[n], tol[n], n)


def test_rows_that_see_nothing_are_zero():
    b, sq, sk, heads, kv, d = 1, 400, 100, 2, 1, 128
    Q, K, V, dO = make(b, sq, sk, heads, kv, d, BF, 3)
    got = run(Q, K, V, dO, b, heads, kv, 30, 2)
    assert (got["O"][:300] == 0).all() and (got["dQ"][:300] == 0).all()
    assert (got["LSE"][:, :, :300] == float("-inf")).all()


@pytest.mark.parametrize("window,sinks", [(300, 4), (5000, 0), (40, 200)])
def test_scores_that_rise_and_fall_by_far(window, sinks):
    """Sharp rows: scores of several hundred, the maximum moving from block to
    block, through the rescaling of O."""
    b, s, heads, kv, d = 1, 900, 2, 1, 128
    Q, K, V, dO = make(b, s, s, heads, kv, d, BF, 4)
    ramp = torch.linspace(-30, 30, s, device="cuda")[:, None]
    u = torch.ones(1, d, device="cuda")
    K = (K.float() * 0.1 + ramp * u * 0.3).to(BF).contiguous()
    Q = (Q.float() * 0.1 + 1.0).to(BF).contiguous()
    got = run(Q, K, V, None, b, heads, kv, window, sinks)
    ref, tol = reference(Q, K, V, b, heads, kv, window, sinks, d ** -0.5)
    # a score's own error grows with its size: 2^-20 of sum |q||k| shifts P by that much
    extra = (tol["LSE"].transpose(1, 2).reshape(s, heads, 1) * 4).expand(s, heads, d)
    close(got["O"], ref["O"], tol["O"] + extra.reshape(s, -1) * V.float().abs().max().double(), "O")
    close(got["LSE"], ref["LSE"], tol["LSE"], "LSE")


def test_scale_argument():
    Q, K, V, dO = make(1, 200, 200, 2, 2, 64, BF, 6)
    got = run(Q, K, V, dO, 1, 2, 2, 50, 1, scale=0.3)
    ref, tol = reference(Q, K, V, 1, 2, 2, 50, 1, 0.3, dO)
    for n in ref:
        close(got[n], ref[n], tol[n], n)


def test_sequences_never_mix():
    """A NaN of one sequence stays in it, whatever tiles its neighbours share."""
    b, s, heads, kv, d = 3, 200, 2, 1, 128
    Q, K, V, dO = make(b, s, s, heads, kv, d, BF, 7)
    a = run(Q, K, V, dO, b, heads, kv, 60, 4)
    K2, V2, Q2, g2 = (x.clone() for x in (K, V, Q, dO))
    for x in (K2, V2, Q2, g2):
        x[s:2 * s] = float("nan")
    c = run(Q2, K2, V2, g2, b, heads, kv, 60, 4)
    for n in ("O", "dQ", "dK", "dV"):
        for rows in (slice(0, s), slice(2 * s, 3 * s)):
            assert torch.equal(a[n][rows], c[n][rows]), n


def test_repeats_bitwise_and_writes_only_its_rows():
    b, s, heads, kv, d = 2, 333, 4, 2, 64
    Q, K, V, dO = make(b, s, s, heads, kv, d, BF, 8)
    a, c = (run(Q, K, V, dO, b, heads, kv, 70, 5) for _ in range(2))
    assert all(torch.equal(a[n], c[n]) for n in a)
    # into the columns of one wider matrix, rows behind and columns beside untouched
    wide = torch.full((b * s + 3, (heads + 2 * kv) * d + 8), 7.0, dtype=BF, device="cuda")
    dQ, dK, dV = (wide[:b * s, i:j] for i, j in ((0, heads * d), (heads * d, (heads + kv) * d),
                                                 ((heads + kv) * d, (heads + 2 * kv) * d)))
    ws = L.window_attn_workspace(b, s, s, heads, kv, d, 70, 5)
    L.tp_window_attn_bwd(Q, K, V, a["O"], a["LSE"], dO, dQ, dK, dV, b, heads, kv, 70, 5, ws)
    assert torch.equal(dQ, a["dQ"]) and torch.equal(dK, a["dK"]) and torch.equal(dV, a["dV"])
    assert (wide[b * s:] == 7).all() and (wide[:, (heads + 2 * kv) * d:] == 7).all()


def test_gradients_against_differences():
    """Directional derivatives of sum(O * w) by central differences of fp64."""
    b, s, heads, kv, d = 1, 150, 2, 1, 64
    Q, K, V, w = make(b, s, s, heads, kv, d, FP, 9)
    got = run(Q, K, V, w, b, heads, kv, 40, 3)

    def loss(q, k, v):
        out, _ = reference64(q, k, v)
        return (out * w.double().reshape(s, heads, d)).sum().item()

    def reference64(q, k, v):
        seen = visible(s, s, 40, 3)
        z = torch.einsum("rhd,cd->hrc", q.reshape(s, heads, d), k) * d ** -0.5
        P = torch.softmax(z.masked_fill(~seen, float("-inf")), -1)
        return torch.einsum("hrc,cd->rhd", P, v), P

    g = torch.Generator(device="cuda").manual_seed(1)
    x = [t.double() for t in (Q, K, V)]
    for i, n in enumerate(("dQ", "dK", "dV")):
        u = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, dn = (loss(*[t + e * u if j == i else t for j, t in enumerate(x)])
                  for e in (1e-4, -1e-4))
        fd, an = (up - dn) / 2e-4, (got[n].double() * u).sum().item()
        # s * heads * d values of about 2^-11 relative error each, random signs
        assert abs(fd - an) <= 2.0 ** -10 * (got[n].double() * u).norm().item() + 1e-6 * abs(fd), n


def test_graph_replay_and_side_stream():
    b, s, heads, kv, d = 1, 1000, 8, 1, 128
    Q, K, V, dO = make(b, s, s, heads, kv, d, BF, 10)
    ws = L.window_attn_workspace(b, s, s, heads, kv, d, 100, 4)
    ref = run(Q, K, V, dO, b, heads, kv, 100, 4, ws=ws)
    out = {n: torch.empty_like(v) for n, v in ref.items()}
    torch.cuda.synchronize()

    def step():
        L.tp_window_attn_fwd(Q, K, V, out["O"], out["LSE"], b, heads, kv, 100, 4)
        L.tp_window_attn_bwd(Q, K, V, out["O"], out["LSE"], dO, out["dQ"], out["dK"], out["dV"], b,
                             heads, kv, 100, 4, ws)

    st = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # both on one workspace
    for g in graphs:
        with torch.cuda.stream(st):
            with torch.cuda.graph(g, stream=st):
                step()
    for g in graphs + graphs:
        for v in out.values():
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], ref[n]) for n in ref)


def test_matches_the_full_causal_core():
    """A window over everything equals tp_attn_fwd's core on the same fp16 QKV."""
    b, s, heads, d = 2, 320, 4, 128
    h = heads * d
    g = torch.Generator(device="cuda").manual_seed(11)
    X, Wqkv, Wo = rn(g, b * s, h), rn(g, h, 3 * h, std=0.05), rn(g, h, h, std=0.05)
    Z, O = torch.empty_like(X), torch.empty_like(X)
    QKV = torch.empty(b * s, 3 * h, dtype=FP, device="cuda")
    LSE = torch.empty(b, heads, s, device="cuda")
    L.tp_attn_fwd(X, Wqkv, Wo, Z, QKV, O, LSE, b, s, heads, 2, True,
                  L.workspace(L.TP_OP_ATTN_FWD, b * s, h, 0, heads, 2, L.TP_BF16))
    got = run(QKV[:, :h], QKV[:, h:2 * h], QKV[:, 2 * h:], None, b, heads, heads, s, 0)
    # the same products; O rounded to fp16 here, to bf16 there
    assert (got["O"].float() - O.float()).abs().max() <= 2.0 ** -8 * O.float().abs().max() * 1.01
    assert (got["LSE"] - LSE).abs().max() <= 1e-5


# ---------------------------------------------------------------- single tokens
def decode_ref(Q, K, V, lens, heads, kv, window, sinks):
    b, cap, d = K.shape[0], K.shape[1], Q.shape[1] // heads
    dt, hs = Q.dtype, half_step(Q.dtype)
    O = torch.zeros(b, heads, d, dtype=torch.float64, device="cuda")
    eO = torch.zeros_like(O)
    lse = torch.full((b, heads), float("-inf"), dtype=torch.float64, device="cuda")
    tl = torch.zeros_like(lse)
    for i, n in enumerate(lens.tolist()):
        n = min(max(n, 0), cap)
        if n == 0:
            continue
        seen = visible(1, n, window, sinks)[0]
        q = Q[i].double().reshape(heads, d)
        k, v = (x[i, :n][seen].double().reshape(-1, kv, d).repeat_interleave(heads // kv, 1)
                for x in (K, V))
        s = torch.einsum("hd,chd->hc", q, k) * d ** -0.5
        P = torch.softmax(s, 1)
        O[i], mag = torch.einsum("hc,chd->hd", P, v), torch.einsum("hc,chd->hd", P, v.abs())
        eO[i] = (hs + F32) * mag + hs * O[i].abs() + (2.0 ** -24 if dt == FP else 0)
        lse[i] = torch.logsumexp(s, 1)
        tl[i] = 2.0 ** -20 * (1 + torch.einsum("hd,chd->hc", q.abs(), k.abs()).amax(1) * d ** -0.5)
    return O.reshape(b, -1), eO.reshape(b, -1), lse, tl


DECODE = [  # b, cap, heads, kv_heads, d, window, sinks, dtype, lens
    (1, 1, 1, 1, 64, 1, 0, BF, [1]),
    (6, 40, 4, 2, 128, 16, 3, BF, [0, 1, 15, 16, 17, 40]),
    (3, 700, 24, 1, 128, 700, 0, FP, [700, 64, 65]),     # 24 heads on one key head: two passes
    (4, 3000, 16, 1, 64, 100, 4, BF, [3000, 104, 103, 2999]),
    (2, 5000, 3, 3, 128, 5000, 0, BF, [4999, 257]),
    (1, 40000, 8, 2, 64, 40000, 0, FP, [39999]),         # many slices
    (5, 900, 10, 2, 128, 300, 64, BF, [900, 1200, -4, 364, 365]),  # clamped to [0, cap]
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "b%dc%dh%d_%dd%dw%ds%d" % c[:7])
def test_decode(case):
    b, cap, heads, kv, d, window, sinks, dt, lens = case
    g = torch.Generator(device="cuda").manual_seed(b + cap)
    Q = rn(g, b, heads * d + 8, dt=dt)[:, :heads * d]
    KV = rn(g, b, cap, 2 * kv * d, dt=dt)
    K, V = KV[:, :, :kv * d], KV[:, :, kv * d:]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for i, m in enumerate(lens):  # whatever lies past a sequence's keys
        KV[i, max(0, m):] = float("nan")
    O = torch.full((b, heads * d), float("nan"), dtype=dt, device="cuda")
    LSE = torch.full((b, heads), float("nan"), device="cuda")
    ws = L.window_attn_decode_workspace(b, cap, heads, kv, d, window, sinks)
    ws.fill_(0xff)
    L.tp_window_attn_decode(Q, K, V, n, O, LSE, heads, kv, window, sinks, ws)
    ref, eO, lse, tl = decode_ref(Q, K, V, n, heads, kv, window, sinks)
    close(O, ref, eO, "O")
    close(LSE, lse, tl, "LSE")
    O2 = torch.empty_like(O)
    L.tp_window_attn_decode(Q, K, V, n, O2, None, heads, kv, window, sinks, ws)
    assert torch.equal(O, O2)


def test_decode_equals_the_last_row_of_the_prompt():
    b, s, heads, kv, d = 2, 777, 8, 2, 128
    Q, K, V, _ = make(b, s, s, heads, kv, d, BF, 12)
    full = run(Q, K, V, None, b, heads, kv, 200, 4)
    last = lambda x: x.reshape(b, s, -1)[:, -1].contiguous()
    O = torch.empty(b, heads * d, dtype=BF, device="cuda")
    lens = torch.full((b,), s, dtype=torch.int32, device="cuda")
    L.tp_window_attn_decode(last(Q), K.reshape(b, s, -1) if K.is_contiguous() else
                            K.contiguous().reshape(b, s, -1), V.contiguous().reshape(b, s, -1),
                            lens, O, None, heads, kv, 200, 4,
                            L.window_attn_decode_workspace(b, s, heads, kv, d, 200, 4))
    ref = last(full["O"]).float()
    # both round P and O to bf16: two half steps each of the row's largest |V|
    assert (O.float() - ref).abs().max() <= 4 * 2.0 ** -8 * V.float().abs().max() * 0.5


def test_decode_replays_with_lengths_that_grow():
    b, cap, heads, kv, d = 3, 600, 4, 1, 64
    g = torch.Generator(device="cuda").manual_seed(13)
    Q, K, V = rn(g, b, heads * d), rn(g, b, cap, d), rn(g, b, cap, d)
    lens = torch.tensor([5, 300, 590], dtype=torch.int32, device="cuda")
    O = torch.empty_like(Q)
    ws = L.window_attn_decode_workspace(b, cap, heads, kv, d, 128, 4)
    call = lambda: L.tp_window_attn_decode(Q, K, V, lens, O, None, heads, kv, 128, 4, ws)
    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for _ in range(3):
        lens += 3
        gr.replay()
        ref, eO, _, _ = decode_ref(Q, K, V, lens, heads, kv, 128, 4)
        close(O, ref, eO, "O")


def test_binding_refuses_mismatched_tensors():
    Q, K, V, dO = make(1, 64, 64, 2, 1, 64, BF, 14)
    O, LSE = torch.empty(64, 128, dtype=BF, device="cuda"), torch.empty(1, 2, 64, device="cuda")
    ok = [Q, K, V, O, LSE, 1, 2, 1, 16, 0]
    L.tp_window_attn_fwd(*ok)
    for i, bad in ((0, Q.float()), (1, K.half()), (1, K[:, :32]), (2, V[:60]), (3, O[:, :64]),
                   (4, LSE.double()), (4, LSE[:, :, :3]), (5, 3), (6, 3), (1, K.cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises((ValueError, L.TPError)):
            L.tp_window_attn_fwd(*args)
    lens = torch.ones(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        L.tp_window_attn_decode(Q[:2], K[:2].reshape(2, 1, 64), V[:2].reshape(2, 1, 64), lens,
                                O[:2], None, 2, 1, 4, 0, torch.empty(256, dtype=torch.uint8,
                                                                    device="cuda"))


@pytest.mark.parametrize("case,std", [
    ((7, 300, 170, 32, 4, 128, 40, 2, BF), 1.0),    # first 130 queries see nothing
    ((6, 333, 333, 40, 8, 64, 100, 3, FP), 6.0),    # late maxima
    ((3, 600, 130, 64, 8, 64, 500, 0, BF), 1.0),    # a whole tile sees nothing
    ((40, 130, 130, 16, 16, 128, 7, 0, BF), 6.0)],
    ids=lambda c: str(c[0]) if isinstance(c, tuple) else None)
def test_several_items_per_block(case, std):
    """More (sequence, head, query tiles) than SMs, so every block takes several,
    into columns and rows of a larger buffer that stays as it was around them."""
    b, sq, sk, heads, kv, d, window, sinks, dt = case
    Q, K, V, dO = make(b, sq, sk, heads, kv, d, dt, seed=5, std=std)
    out = run(Q, K, V, dO, b, heads, kv, window, sinks)
    ref, tol = reference(Q, K, V, b, heads, kv, window, sinks, d ** -0.5, dO)
    for n in out:
        close(out[n], ref[n], tol[n], n)
    big = torch.full((b * sq + 5, heads * d + 72), 7.0, dtype=dt, device="cuda")
    view = big[2:2 + b * sq, 64:64 + heads * d]
    LSE = torch.empty(b, heads, sq, device="cuda")
    L.tp_window_attn_fwd(Q, K, V, view, LSE, b, heads, kv, window, sinks)
    assert torch.equal(view, out["O"]) and torch.equal(LSE, out["LSE"])
    view.fill_(7.0)
    assert bool((big == 7.0).all())


@pytest.mark.parametrize("dt", [BF, FP])
def test_decode_of_few_outputs_rounds_once(dt):
    """Up to 8192 outputs P has two terms, so O is off by its own rounding and the
    fp32 parts of `reference` (2 hs^2 of P |V| is what two terms leave; for fp16
    half its smallest step per key)."""
    b, cap, heads, kv, d = 2, 700, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(12)
    Q, K, V = rn(g, b, heads * d, dt=dt), rn(g, b, cap, kv * d, dt=dt), rn(g, b, cap, kv * d, dt=dt)
    lens = torch.full((b,), cap, dtype=torch.int32, device="cuda")
    O, ws = torch.empty_like(Q), L.window_attn_decode_workspace(b, cap, heads, kv, d, 400, 3)
    L.tp_window_attn_decode(Q, K, V, lens, O, None, heads, kv, 400, 3, ws)
    ref, _ = reference(Q, K.reshape(b * cap, -1), V.reshape(b * cap, -1), b, heads, kv, 400, 3,
                       d ** -0.5)
    big, _ = reference(Q, K.reshape(b * cap, -1), V.abs().reshape(b * cap, -1), b, heads, kv, 400,
                       3, d ** -0.5)
    hs = half_step(dt)
    tiny = 403 * 2.0 ** -25 * V.abs().max().double() if dt == FP else 0.0
    tol = hs * ref["O"].abs() + (F32 + 2 * hs * hs) * big["O"] + tiny
    close(O, ref["O"], tol, "O")
