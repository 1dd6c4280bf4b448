"""The decoder-layer operators run together: projection, query/key norm with
rotary positions, windowed attention, output projection, gated block.

    QKV = X Wqkv;  Q, K = rotary(norm(Q, K));  X1 = X + Attn(Q, K, V) Wo;
    X2 = X1 + GLU(X1)

Tolerances: normwise, from the bf16 roundings in a row (1.7e-3 each, see
parity.py's 5e-3 for up to eight of them added in squares).  X2 passes through
eight (QKV, Q/K, P, O, the projection, X1, H, Z).  The longest gradient, gq's,
meets twenty: QKV as q, k and v, Qr, Kr, P, O, the projection, X1, G, U, [dG |
dU], dX1 twice, dO, P and dS, dQr, dQ and its own: sqrt(20) * 1.7e-3 = 7.6e-3.
That is the root mean square; the norm of n independent errors scatters about
it by a relative 1 / sqrt(2 n), and the norm weights have only n = 64 values,
so four such deviations are allowed: 7.6e-3 * (1 + 4 / sqrt(2 n)).
"""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
B, S, H, KV, D, F, W, SINK = 2, 300, 8, 2, 64, 1408, 70, 3
HID, NQ, NK = 512, H * D, KV * D
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


def params(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g, device="cuda") * std
                                        + mean).to(BF)
    return dict(X=rn(B * S, HID), Wqkv=rn(HID, NQ + 2 * NK, std=HID ** -0.5),
                gq=rn(D, std=0.1, mean=1.0), gk=rn(D, std=0.1, mean=1.0),
                Wo=rn(NQ, HID, std=NQ ** -0.5), Wgu=rn(HID, 2 * F, std=HID ** -0.5),
                Wd=rn(F, HID, std=F ** -0.5)), rn(B * S, HID)


def side(n_rows=S):
    pos = torch.arange(n_rows, dtype=torch.int32, device="cuda").repeat(B)
    fr = torch.pow(10000.0, -torch.arange(D // 2, dtype=torch.float64, device="cuda") * 2 / D)
    return pos, fr


def forward(p, pos, fr):
    new = lambda *s: torch.empty(*s, dtype=BF, device="cuda")
    X = p["X"]
    QKV = new(B * S, NQ + 2 * NK)
    L.tp_linear_col(X, p["Wqkv"], None, QKV, 1)
    Q, K, V = QKV[:, :NQ], QKV[:, NQ:NQ + NK], QKV[:, NQ + NK:]
    Qr, Kr, O, A, Z = new(B * S, NQ), new(B * S, NK), new(B * S, NQ), new(B * S, HID), new(B * S, HID)
    L.tp_qk_norm_rope_fwd(Q, K, p["gq"], p["gk"], pos, fr, Qr, Kr, D, True, False, EPS)
    LSE = torch.empty(B, H, S, device="cuda")
    L.tp_window_attn_fwd(Qr, Kr, V, O, LSE, B, H, KV, W, SINK)
    L.tp_linear_row(O, p["Wo"], None, A, 1)
    X1 = X + A
    GU = torch.empty(B * S, 2 * F, dtype=torch.float16, device="cuda")
    L.tp_glu_fwd(X1, p["Wgu"], None, p["Wd"], None, Z, GU, 1, L.TP_ACT_SILU,
                 L.workspace(L.TP_OP_GLU_FWD, B * S, HID, F, 0, 1, L.TP_BF16))
    return X1 + Z, dict(QKV=QKV, Q=Q, K=K, V=V, Qr=Qr, Kr=Kr, O=O, LSE=LSE, X1=X1, GU=GU)


def backward(p, s, dX2, pos, fr):
    new = torch.empty_like
    dX1, dWgu, dWd = new(s["X1"]), new(p["Wgu"]), new(p["Wd"])
    L.tp_glu_bwd(s["X1"], p["Wgu"], None, p["Wd"], s["GU"], dX2, dX1, dWgu, None, dWd, None, 1,
                 L.TP_ACT_SILU, L.workspace(L.TP_OP_GLU_BWD, B * S, HID, F, 0, 1, L.TP_BF16))
    dX1 += dX2
    dO = dX1 @ p["Wo"].t()
    dQKV = new(s["QKV"])
    dQ, dK, dV = dQKV[:, :NQ], dQKV[:, NQ:NQ + NK], dQKV[:, NQ + NK:]
    dQr, dKr = new(s["Qr"]), new(s["Kr"])
    L.tp_window_attn_bwd(s["Qr"], s["Kr"], s["V"], s["O"], s["LSE"], dO, dQr, dKr, dV, B, H, KV, W,
                         SINK, L.window_attn_workspace(B, S, S, H, KV, D, W, SINK))
    dgq, dgk = new(p["gq"]), new(p["gk"])
    L.tp_qk_norm_rope_bwd(s["Q"], s["K"], p["gq"], p["gk"], pos, fr, dQr, dKr, dQ, dK, dgq, dgk, D,
                          L.qk_norm_rope_workspace(B * S, D), True, False, EPS)
    return dict(X=dX1 + dQKV @ p["Wqkv"].t(), Wqkv=p["X"].t() @ dQKV, gq=dgq, gk=dgk,
                Wo=s["O"].t() @ dX1, Wgu=dWgu, Wd=dWd)


def reference(p, pos, fr):
    def head(x, g):
        y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * g
        t = pos.double()[:, None] * fr
        c, sn = t.cos()[:, None], t.sin()[:, None]
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat([a * c - b * sn, b * c + a * sn], -1)

    M = p["X"].shape[0]
    qkv = p["X"] @ p["Wqkv"]
    q = head(qkv[:, :NQ].reshape(M, H, D), p["gq"]).reshape(B, S, H, D)
    k = head(qkv[:, NQ:NQ + NK].reshape(M, KV, D), p["gk"]).reshape(B, S, KV, D)
    v = qkv[:, NQ + NK:].reshape(B, S, KV, D)
    k, v = k.repeat_interleave(H // KV, 2), v.repeat_interleave(H // KV, 2)
    r = torch.arange(S, device="cuda")
    gap = r[:, None] - r[None, :]
    seen = (gap >= 0) & ((gap < W) | (r[None, :] < SINK))
    z = torch.einsum("brhd,bchd->bhrc", q, k) * D ** -0.5
    o = torch.einsum("bhrc,bchd->brhd",
                     torch.softmax(z.masked_fill(~seen, float("-inf")), -1), v).reshape(M, NQ)
    x1 = p["X"] + o @ p["Wo"]
    gu = x1 @ p["Wgu"]
    g, u = gu[:, :F], gu[:, F:]
    return x1 + (g * torch.sigmoid(g) * u) @ p["Wd"]


def normwise(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def test_training_step():
    p, dX2 = params()
    pos, fr = side()
    X2, saves = forward(p, pos, fr)
    grads = backward(p, saves, dX2, pos, fr)
    p64 = {n: v.double().requires_grad_() for n, v in p.items()}
    ref = reference(p64, pos, fr)
    rg = dict(zip(p64, torch.autograd.grad(ref, list(p64.values()), dX2.double())))
    assert normwise(X2, ref.detach()) <= 5e-3
    for n in rg:
        nw = normwise(grads[n], rg[n])
        assert nw <= 7.6e-3 * (1 + 4 / (2 * rg[n].numel()) ** 0.5), (n, nw)


def test_generation_follows_the_prompt():
    """Token by token over a cache against the prompt's rows: norm and rotation
    of the new token in place, keys and values appended, one query each."""
    p, _ = params(1)
    pos, fr = side()
    X2, s = forward(p, pos, fr)
    n0, steps = 290, 10
    shape = lambda x: x.reshape(B, S, -1)
    Kc = torch.full((B, 512, NK), float("nan"), dtype=BF, device="cuda")
    Vc = Kc.clone()
    Kc[:, :n0], Vc[:, :n0] = shape(s["Kr"])[:, :n0], shape(s["V"])[:, :n0]
    lens = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    wsd = L.window_attn_decode_workspace(B, 512, H, KV, D, W, SINK)
    wsg = L.workspace(L.TP_OP_GLU_FWD, B, HID, F, 0, 1, L.TP_BF16)
    new = lambda n: torch.empty(B, n, dtype=BF, device="cuda")
    for i in range(n0, n0 + steps):
        x = shape(p["X"])[:, i].contiguous()
        qkv, O, A, Z = new(NQ + 2 * NK), new(NQ), new(HID), new(HID)
        L.tp_linear_col(x, p["Wqkv"], None, qkv, 1)
        q, k = qkv[:, :NQ], qkv[:, NQ:NQ + NK]
        L.tp_qk_norm_rope_fwd(q, k, p["gq"], p["gk"], lens, fr, q, k, D, True, False, EPS)
        Kc[:, i], Vc[:, i] = k, qkv[:, NQ + NK:]
        lens += 1
        L.tp_window_attn_decode(q, Kc, Vc, lens, O, None, H, KV, W, SINK, wsd)
        L.tp_linear_row(O, p["Wo"], None, A, 1)
        x1 = x + A
        L.tp_glu_fwd(x1, p["Wgu"], None, p["Wd"], None, Z, None, 1, L.TP_ACT_SILU, wsg)
        # both sides carry the same roundings, each within 5e-3 of the exact row
        assert normwise(x1 + Z, shape(X2)[:, i].double()) <= 1e-2, i


def test_a_captured_step_beside_an_eager_one():
    """The training step captured in a graph while an eager step's saves live."""
    p, dX2 = params(2)
    pos, fr = side()
    X2, saves = forward(p, pos, fr)
    grads = backward(p, saves, dX2, pos, fr)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        forward(p, pos, fr)  # warm the side stream's allocator and library handles
        backward(p, saves, dX2, pos, fr)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            Y2, s2 = forward(p, pos, fr)
            g2 = backward(p, s2, dX2, pos, fr)
    g.replay()
    again = backward(p, saves, dX2, pos, fr)
    torch.cuda.synchronize()
    assert torch.equal(Y2, X2)
    for n in ("Wgu", "Wd", "gq", "gk"):
        assert torch.equal(g2[n], grads[n]) and torch.equal(again[n], grads[n]), n
