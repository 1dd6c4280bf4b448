"""Cases for the decoder-layer operators: query/key norm with rotary positions,
sliding-window attention with sinks (prompt, training, single token over a
cache) and the gated feed-forward block.

run() makes one pass through an operator.  With `own` false it computes the
operator's plain form (elementary torch operations in fp32, angles in fp64,
rounded once at the end); with `own` true it makes the calls a user makes of
megatron_tensor_transformer_logical_b200.binding.  exact() computes the same
outputs in fp64 from the definitions, through autograd.

Definitions, per operator:

qk_norm_rope   x a head's row of d values: x^ = x / sqrt(mean(x^2) + eps) * g
               (RMS norm, weight g [d] shared by the heads), then the first
               d_rot values are rotated in pairs by the angle pos * inv_freq[i]:
               (a, b) -> (a cos - b sin, b cos + a sin), the pairs being
               (i, i + d_rot / 2) or, interleaved, (2 i, 2 i + 1).
window         query r of a sequence sits at position p = r + sk - sq; key c is
               visible when c <= p and (p - c < window or c < sinks);
               O = softmax(scale Q K^T over the visible keys) V, query head j
               reading key / value head j * kv_heads / heads.
decode         one query per sequence at position lens[i] - 1 of a cache.
glu            Z = (act(X Wg + bg) * (X Wu + bu)) Wd + bd, Wgu = [Wg | Wu].
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rope(name, M, heads, kv_heads, d, d_rot, dtype, train, max_pos, interleaved=False):
    return dict(name=name, op="rope", M=M, heads=heads, kv_heads=kv_heads, d=d, d_rot=d_rot,
                dtype=dtype, train=train, max_pos=max_pos, interleaved=interleaved)


def _window(name, b, sq, sk, heads, kv_heads, d, window, sinks, dtype, train):
    return dict(name=name, op="window", b=b, sq=sq, sk=sk, heads=heads, kv_heads=kv_heads, d=d,
                window=window, sinks=sinks, dtype=dtype, train=train)


def _decode(name, b, cap, heads, kv_heads, d, window, sinks, dtype):
    return dict(name=name, op="decode", b=b, cap=cap, heads=heads, kv_heads=kv_heads, d=d,
                window=window, sinks=sinks, dtype=dtype)


def _glu(name, M, h, f, t, act, bias, train):
    return dict(name=name, op="glu", M=M, h=h, f=f, t=t, act=act, bias=bias, train=train)


def listed():
    return [
        # one decoding step of 4 sequences deep in their contexts: pure latency
        _rope("rope_token", 4, 32, 8, 128, 128, "bf16", False, 131072),
        # a training step's 8192 tokens, grouped key heads
        _rope("rope_train", 8192, 32, 8, 128, 128, "bf16", True, 4096),
        # a ragged prompt in fp16, small heads, half of each head rotated, interleaved pairs
        _rope("rope_ragged", 3001, 20, 20, 64, 32, "fp16", False, 32768, True),
        # full-precision training of a small model
        _rope("rope_fp32", 2050, 16, 4, 96, 96, "fp32", True, 2048),
        # a long prompt, window of 1024 and four sinks
        _window("window_prompt", 1, 8192, 8192, 32, 8, 128, 1024, 4, "bf16", False),
        # a training step, two sequences of 4096
        _window("window_train", 2, 4096, 4096, 32, 8, 128, 1024, 4, "bf16", True),
        # training on odd lengths, one key head per query head, fp16, no sinks
        _window("window_ragged", 3, 1931, 1931, 12, 12, 64, 257, 0, "fp16", True),
        # one decoding step of a full batch over a windowed cache
        _decode("decode_batch", 32, 8192, 32, 8, 128, 4096, 4, "bf16"),
        # one decoding step of one sequence that sees its whole long context
        _decode("decode_long", 1, 131072, 32, 4, 128, 131072, 0, "bf16"),
        # one token through a gated feed-forward block: reading the weights
        _glu("glu_token", 1, 4096, 14336, 1, "silu", False, False),
        # an odd decoding batch, biases, the erf GeLU
        _glu("glu_batch", 13, 2048, 5632, 4, "gelu", True, False),
        # a training step's forward and backward
        _glu("glu_train", 4096, 4096, 14336, 8, "silu", False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "window", "window", "decode", "decode", "glu", "glu"])
    if kind == "rope":
        d = rng.choice([64, 80, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 8])
        tokens = _log(rng, 1, 8192 * 40 * 128 // (kv * (group + 1) * d))
        d_rot = rng.choice([d, d, 16 * max(1, d // 32)])
        c = _rope(None, min(tokens, 16384), kv * group, kv, d, d_rot,
                  rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.random() < 0.5,
                  _log(rng, 128, 1 << 20), rng.random() < 0.3)
        if c["dtype"] == "fp32":
            c["M"] = max(1, c["M"] // 2)
    elif kind == "window":
        d = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4])
        train = rng.random() < 0.5
        b = rng.choice([1, 1, 2, 3])
        sk = _log(rng, 16, 4096)
        sq = sk if rng.random() < 0.7 else rng.randint(1, sk)
        c = _window(None, b, sq, sk, kv * group, kv, d, _log(rng, 16, 4096),
                    rng.choice([0, 0, 1, 4, 64, 130]), rng.choice(["bf16", "bf16", "fp16"]), train)
    elif kind == "decode":
        d = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 8, 16])
        b = _log(rng, 1, 48)
        cap = _log(rng, 16, min(131072, (1 << 28) // (b * kv * d)))
        c = _decode(None, b, cap, kv * group, kv, d, rng.choice([_log(rng, 1, cap), cap]),
                    rng.choice([0, 1, 4, 64]), rng.choice(["bf16", "bf16", "fp16"]))
    else:
        t = rng.choice([1, 1, 2, 4, 8])
        h = 8 * _log(rng, 16, 512)
        f = 8 * t * max(1, _log(rng, 32, 1536) // t)
        train = rng.random() < 0.4
        c = _glu(None, _log(rng, 1, 3000), h, f, t, rng.choice(["silu", "gelu"]),
                 rng.random() < 0.4, train)
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = _gen(seed)
    op = case["op"]
    s = {}
    if op == "rope":
        dt = _DTYPES[case["dtype"]]
        M, d = case["M"], case["d"]
        nq, nk = case["heads"] * d, case["kv_heads"] * d
        # a projection's output [q | k | v]: the operator reads the q and k columns
        qkv = _randn(g, M, nq + 2 * nk, dtype=dt)
        s["Q"], s["K"] = qkv[:, :nq], qkv[:, nq:nq + nk]
        s["gq"] = _randn(g, d, dtype=dt, std=0.1, mean=1.0)
        s["gk"] = _randn(g, d, dtype=dt, std=0.1, mean=1.0)
        s["pos"] = torch.randint(0, case["max_pos"], (M,), generator=g, device="cuda",
                                 dtype=torch.int32)
        i = torch.arange(case["d_rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = torch.pow(500000.0, -2.0 * i / case["d_rot"])
        if case["train"]:
            s["dQo"] = _randn(g, M, nq, dtype=dt)
            s["dKo"] = _randn(g, M, nk, dtype=dt)
    elif op == "window":
        dt = _DTYPES[case["dtype"]]
        b, sq, sk, d = case["b"], case["sq"], case["sk"], case["d"]
        nq, nk = case["heads"] * d, case["kv_heads"] * d
        s["Q"] = _randn(g, b * sq, nq, dtype=dt)
        kv = _randn(g, b * sk, 2 * nk, dtype=dt)
        s["K"], s["V"] = kv[:, :nk], kv[:, nk:]
        if case["train"]:
            s["dO"] = _randn(g, b * sq, nq, dtype=dt)
    elif op == "decode":
        dt = _DTYPES[case["dtype"]]
        b, cap, d = case["b"], case["cap"], case["d"]
        s["Q"] = _randn(g, b, case["heads"] * d, dtype=dt)
        s["Kc"] = _randn(g, b, cap, case["kv_heads"] * d, dtype=dt)
        s["Vc"] = _randn(g, b, cap, case["kv_heads"] * d, dtype=dt)
        lo = max(1, cap // 2) if b > 1 else max(1, cap - cap // 64)
        s["lens"] = torch.randint(lo, cap + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    else:
        dt = torch.bfloat16
        M, h, f = case["M"], case["h"], case["f"]
        s["X"] = _randn(g, M, h, dtype=dt)
        s["Wgu"] = _randn(g, h, 2 * f, dtype=dt, std=h ** -0.5)
        s["Wd"] = _randn(g, f, h, dtype=dt, std=f ** -0.5)
        s["bgu"] = _randn(g, 2 * f, dtype=dt, std=0.1) if case["bias"] else None
        s["bd"] = _randn(g, h, dtype=dt, std=0.1) if case["bias"] else None
        if case["train"]:
            s["dZ"] = _randn(g, M, h, dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """Output buffers and workspaces, as a user's program keeps them."""
    from megatron_tensor_transformer_logical_b200 import binding as L
    case = s["case"]
    op = case["op"]
    s["L"] = L
    if op == "rope":
        d = case["d"]
        s["Qo"] = torch.empty_like(s["Q"], memory_format=torch.contiguous_format)
        s["Ko"] = torch.empty_like(s["K"], memory_format=torch.contiguous_format)
        if case["train"]:
            s["dQ"], s["dK"] = torch.empty_like(s["dQo"]), torch.empty_like(s["dKo"])
            s["dgq"], s["dgk"] = torch.empty_like(s["gq"]), torch.empty_like(s["gk"])
            s["ws"] = L.qk_norm_rope_workspace(case["M"], d)
    elif op == "window":
        b, sq = case["b"], case["sq"]
        s["O"] = torch.empty_like(s["Q"])
        s["LSE"] = torch.empty(b, case["heads"], sq, dtype=torch.float32, device="cuda")
        if case["train"]:
            s["dQ"] = torch.empty_like(s["Q"])
            s["dK"] = torch.empty_like(s["K"], memory_format=torch.contiguous_format)
            s["dV"] = torch.empty_like(s["V"], memory_format=torch.contiguous_format)
            s["ws"] = L.window_attn_workspace(b, sq, case["sk"], case["heads"], case["kv_heads"],
                                              case["d"], case["window"], case["sinks"])
    elif op == "decode":
        s["O"] = torch.empty_like(s["Q"])
        s["LSE"] = torch.empty(case["b"], case["heads"], dtype=torch.float32, device="cuda")
        s["ws"] = L.window_attn_decode_workspace(case["b"], case["cap"], case["heads"],
                                                 case["kv_heads"], case["d"], case["window"],
                                                 case["sinks"])
    else:
        M, h, f, t = case["M"], case["h"], case["f"], case["t"]
        s["Z"] = torch.empty_like(s["X"])
        s["act"] = L.TP_ACT_SILU if case["act"] == "silu" else L.TP_ACT_GELU
        s["ws"] = L.workspace(L.TP_OP_GLU_FWD, M, h, f, 0, t, L.TP_BF16)
        if case["train"]:
            s["GU"] = torch.empty(M, 2 * f, dtype=torch.float16, device="cuda")
            s["dX"], s["dWgu"] = torch.empty_like(s["X"]), torch.empty_like(s["Wgu"])
            s["dWd"] = torch.empty_like(s["Wd"])
            s["dbgu"] = torch.empty_like(s["bgu"]) if case["bias"] else None
            s["dbd"] = torch.empty_like(s["bd"]) if case["bias"] else None
            s["wsb"] = L.workspace(L.TP_OP_GLU_BWD, M, h, f, 0, t, L.TP_BF16)


# ---------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "window": _own_window, "decode": _own_decode,
                "glu": _own_glu}[op](state)
    return {"rope": _plain_rope, "window": _plain_window, "decode": _plain_decode,
            "glu": _plain_glu}[op](state)


def _own_rope(s):
    L, c = s["L"], s["case"]
    L.tp_qk_norm_rope_fwd(s["Q"], s["K"], s["gq"], s["gk"], s["pos"], s["inv_freq"], s["Qo"],
                          s["Ko"], c["d"], True, c["interleaved"], 1e-6)
    out = {"Q": s["Qo"], "K": s["Ko"]}
    if c["train"]:
        L.tp_qk_norm_rope_bwd(s["Q"], s["K"], s["gq"], s["gk"], s["pos"], s["inv_freq"], s["dQo"],
                              s["dKo"], s["dQ"], s["dK"], s["dgq"], s["dgk"], c["d"], s["ws"],
                              True, c["interleaved"], 1e-6)
        out.update(dQ=s["dQ"], dK=s["dK"], dgq=s["dgq"], dgk=s["dgk"])
    return out


def _own_window(s):
    L, c = s["L"], s["case"]
    L.tp_window_attn_fwd(s["Q"], s["K"], s["V"], s["O"], s["LSE"], c["b"], c["heads"],
                         c["kv_heads"], c["window"], c["sinks"])
    out = {"O": s["O"], "LSE": s["LSE"]}
    if c["train"]:
        L.tp_window_attn_bwd(s["Q"], s["K"], s["V"], s["O"], s["LSE"], s["dO"], s["dQ"], s["dK"],
                             s["dV"], c["b"], c["heads"], c["kv_heads"], c["window"], c["sinks"],
                             s["ws"])
        out.update(dQ=s["dQ"], dK=s["dK"], dV=s["dV"])
    return out


def _own_decode(s):
    L, c = s["L"], s["case"]
    L.tp_window_attn_decode(s["Q"], s["Kc"], s["Vc"], s["lens"], s["O"], s["LSE"], c["heads"],
                            c["kv_heads"], c["window"], c["sinks"], s["ws"])
    return {"O": s["O"], "LSE": s["LSE"]}


def _own_glu(s):
    L, c = s["L"], s["case"]
    L.tp_glu_fwd(s["X"], s["Wgu"], s["bgu"], s["Wd"], s["bd"], s["Z"], s.get("GU"), c["t"],
                 s["act"], s["ws"])
    out = {"Z": s["Z"]}
    if c["train"]:
        L.tp_glu_bwd(s["X"], s["Wgu"], s["bgu"], s["Wd"], s["GU"], s["dZ"], s["dX"], s["dWgu"],
                     s["dbgu"], s["dWd"], s["dbd"], c["t"], s["act"], s["wsb"])
        out.update(dX=s["dX"], dWgu=s["dWgu"], dWd=s["dWd"])
        if c["bias"]:
            out.update(dbgu=s["dbgu"], dbd=s["dbd"])
    return out


# -------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, d_rot, interleaved, sign):
    """x [M, heads, d] with its first d_rot values rotated by sign * angle."""
    r = x[..., :d_rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
    else:
        a, b = r[..., :d_rot // 2], r[..., d_rot // 2:]
    c, t = cos[:, None, :], sign * sin[:, None, :]
    ra, rb = a * c - b * t, b * c + a * t
    y = x.clone()
    if interleaved:
        y[..., 0:d_rot:2], y[..., 1:d_rot:2] = ra, rb
    else:
        y[..., :d_rot // 2], y[..., d_rot // 2:d_rot] = ra, rb
    return y


def _plain_rope(s):
    c = s["case"]
    M, d, dr, il = c["M"], c["d"], c["d_rot"], c["interleaved"]
    ang = s["pos"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    out = {}
    for n in ("Q", "K"):
        dt = s[n].dtype
        x = s[n].float().reshape(M, -1, d)
        g = s["g" + n.lower()].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        xh = x * r
        y = _rotate(xh * g, cos, sin, dr, il, 1.0)
        out[n] = y.reshape(M, -1).to(dt)
        if c["train"]:
            dz = _rotate(s["d" + n + "o"].float().reshape(M, -1, d), cos, sin, dr, il, -1.0)
            out["dg" + n.lower()] = (dz * xh).sum((0, 1)).to(dt)
            dxh = dz * g
            dx = r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
            out["d" + n] = dx.reshape(M, -1).to(dt)
    return out


def _plain_window(s):
    c = s["case"]
    b, sq, sk, d = c["b"], c["sq"], c["sk"], c["d"]
    H, Hk = c["heads"], c["kv_heads"]
    G = H // Hk
    dt = s["Q"].dtype
    scale = d ** -0.5
    p = torch.arange(sq, device="cuda")[:, None] + (sk - sq)
    k = torch.arange(sk, device="cuda")[None, :]
    hidden = ~((k <= p) & ((p - k < c["window"]) | (k < c["sinks"])))
    Q = s["Q"].reshape(b, sq, H, d)
    K, V = (s[n].reshape(b, sk, Hk, d) for n in ("K", "V"))
    O, LSE = torch.empty_like(Q), torch.empty(b, H, sq, device="cuda")
    train = c["train"]
    if train:
        dO = s["dO"].reshape(b, sq, H, d)
        dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    for i in range(b):
        for j in range(Hk):
            hs = slice(j * G, (j + 1) * G)
            q = Q[i, :, hs].float().transpose(0, 1)          # [G, sq, d]
            kk, vv = K[i, :, j].float(), V[i, :, j].float()  # [sk, d]
            z = torch.matmul(q, kk.t()) * scale
            z.masked_fill_(hidden, float("-inf"))
            m = z.amax(-1, keepdim=True)
            e = torch.exp(z - m)
            l = e.sum(-1, keepdim=True)
            P = e / l
            o = torch.matmul(P, vv)
            O[i, :, hs] = o.transpose(0, 1).to(dt)
            LSE[i, hs] = (m + torch.log(l))[..., 0]
            if train:
                g = dO[i, :, hs].float().transpose(0, 1)
                dP = torch.matmul(g, vv.t())
                dS = P * (dP - (g * o).sum(-1, keepdim=True)) * scale
                dQ[i, :, hs] = torch.matmul(dS, kk).transpose(0, 1).to(dt)
                dK[i, :, j] = torch.matmul(dS.transpose(1, 2), q).sum(0).to(dt)
                dV[i, :, j] = torch.matmul(P.transpose(1, 2), g).sum(0).to(dt)
    out = {"O": O.reshape(b * sq, H * d), "LSE": LSE}
    if train:
        out.update(dQ=dQ.reshape(b * sq, H * d), dK=dK.reshape(b * sk, Hk * d),
                   dV=dV.reshape(b * sk, Hk * d))
    return out


def _plain_decode(s):
    c = s["case"]
    b, cap, d, H, Hk = c["b"], c["cap"], c["d"], c["heads"], c["kv_heads"]
    q = s["Q"].float().reshape(b, Hk, H // Hk, d)
    k = s["Kc"].float().reshape(b, cap, Hk, d).permute(0, 2, 3, 1)
    z = torch.matmul(q, k) * d ** -0.5
    pos = torch.arange(cap, device="cuda")[None, :]
    p = s["lens"].long()[:, None] - 1
    hidden = ~((pos <= p) & ((p - pos < c["window"]) | (pos < c["sinks"])))
    z.masked_fill_(hidden[:, None, None, :], float("-inf"))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    v = s["Vc"].float().reshape(b, cap, Hk, d).permute(0, 2, 1, 3)
    o = torch.matmul(e, v) / l
    return {"O": o.reshape(b, H * d).to(s["Q"].dtype), "LSE": (m + torch.log(l)).reshape(b, H)}


def _act(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-x))
        return x * sg, sg * (1.0 + x * (1.0 - sg))
    cdf = 0.5 * (1.0 + torch.erf(x * 0.7071067811865476))
    return x * cdf, cdf + x * torch.exp(-0.5 * x * x) * 0.3989422804014327


def _plain_glu(s):
    c = s["case"]
    f = c["f"]
    dt = s["X"].dtype
    X, Wgu, Wd = s["X"].float(), s["Wgu"].float(), s["Wd"].float()
    GU = torch.matmul(X, Wgu)
    if c["bias"]:
        GU = GU + s["bgu"].float()
    a, da = _act(GU[:, :f], c["act"])
    U = GU[:, f:]
    H = a * U
    Z = torch.matmul(H, Wd)
    if c["bias"]:
        Z = Z + s["bd"].float()
    out = {"Z": Z.to(dt)}
    if c["train"]:
        dZ = s["dZ"].float()
        dH = torch.matmul(dZ, Wd.t())
        dGU = torch.cat([dH * U * da, dH * a], 1)
        out["dX"] = torch.matmul(dGU, Wgu.t()).to(dt)
        out["dWgu"] = torch.matmul(X.t(), dGU).to(dt)
        out["dWd"] = torch.matmul(H.t(), dZ).to(dt)
        if c["bias"]:
            out["dbgu"], out["dbd"] = dGU.sum(0).to(dt), dZ.sum(0).to(dt)
    return out


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = _inputs(case, seed)
    return {"rope": _exact_rope, "window": _exact_window, "decode": _exact_decode,
            "glu": _exact_glu}[case["op"]](case, s)


def _exact_rope(c, s):
    M, d, dr = c["M"], c["d"], c["d_rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None] * s["inv_freq"])
    out = {}
    for n in ("Q", "K"):
        x = s[n].double().reshape(M, -1, d).requires_grad_()
        g = s["g" + n.lower()].double().requires_grad_()
        y = x / (x.square().sum(-1, keepdim=True) / d + 1e-6).sqrt() * g
        r, rest = y[..., :dr], y[..., dr:]
        pairs = r.unflatten(-1, (dr // 2, 2)) if c["interleaved"] else \
            r.unflatten(-1, (2, dr // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        y = torch.cat([z, rest], -1).reshape(M, -1)
        out[n] = y.detach()
        if c["train"]:
            dx, dg = torch.autograd.grad(y, (x, g), s["d" + n + "o"].double())
            out["d" + n], out["dg" + n.lower()] = dx.reshape(M, -1), dg
    order = ["Q", "K"] + (["dQ", "dK", "dgq", "dgk"] if c["train"] else [])
    return {k: out[k] for k in order}


def _exact_window(c, s):
    b, sq, sk, d, H, Hk = c["b"], c["sq"], c["sk"], c["d"], c["heads"], c["kv_heads"]
    f64 = dict(dtype=torch.float64, device="cuda")
    O, LSE = torch.empty(b, sq, H, d, **f64), torch.empty(b, H, sq, **f64)
    grads = {"dQ": torch.zeros(b, sq, H, d, **f64), "dK": torch.zeros(b, sk, Hk, d, **f64),
             "dV": torch.zeros(b, sk, Hk, d, **f64)}
    Q = s["Q"].reshape(b, sq, H, d)
    K, V = s["K"].reshape(b, sk, Hk, d), s["V"].reshape(b, sk, Hk, d)
    step = 512
    for i in range(b):
        for h in range(H):
            kh = h * Hk // H
            for r0 in range(0, sq, step):
                r1 = min(r0 + step, sq)
                p = torch.arange(r0, r1, device="cuda") + (sk - sq)
                lo = max(0, r0 + sk - sq - c["window"] + 1)
                hi = r1 + sk - sq
                # the keys any of these queries sees, in order
                cols = torch.cat([torch.arange(0, min(lo, c["sinks"], hi), device="cuda"),
                                  torch.arange(lo, hi, device="cuda")])
                q = Q[i, r0:r1, h].double().requires_grad_()
                k = K[i, cols, kh].double().requires_grad_()
                v = V[i, cols, kh].double().requires_grad_()
                gap = p[:, None] - cols[None, :]
                seen = (gap >= 0) & ((gap < c["window"]) | (cols[None, :] < c["sinks"]))
                z = torch.einsum("rd,cd->rc", q, k) / math.sqrt(d)
                z = torch.where(seen, z, torch.full_like(z, float("-inf")))
                lse = torch.logsumexp(z, 1)
                o = torch.einsum("rc,cd->rd", torch.exp(z - lse[:, None]), v)
                O[i, r0:r1, h], LSE[i, h, r0:r1] = o.detach(), lse.detach()
                if c["train"]:
                    g = s["dO"].reshape(b, sq, H, d)[i, r0:r1, h].double()
                    gq, gk, gv = torch.autograd.grad(o, (q, k, v), g)
                    grads["dQ"][i, r0:r1, h] = gq
                    grads["dK"][i, :, kh].index_add_(0, cols, gk)
                    grads["dV"][i, :, kh].index_add_(0, cols, gv)
    out = {"O": O.reshape(b * sq, -1), "LSE": LSE}
    if c["train"]:
        out.update({n: g.reshape(b * g.shape[1], -1) for n, g in grads.items()})
    return out


def _exact_decode(c, s):
    b, d, H, Hk = c["b"], c["d"], c["heads"], c["kv_heads"]
    G = H // Hk
    O, LSE = [], []
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"])
        cols = torch.cat([torch.arange(0, min(lo, c["sinks"]), device="cuda"),
                          torch.arange(lo, n, device="cuda")])
        k = s["Kc"][i, cols].double().reshape(-1, Hk, d)
        v = s["Vc"][i, cols].double().reshape(-1, Hk, d)
        q = s["Q"][i].double().reshape(Hk, G, d)
        z = torch.einsum("hgd,chd->hgc", q, k) / math.sqrt(d)
        O.append(torch.einsum("hgc,chd->hgd", torch.softmax(z, -1), v).reshape(-1))
        LSE.append(torch.logsumexp(z, -1).reshape(-1))
    return {"O": torch.stack(O), "LSE": torch.stack(LSE)}


def _exact_glu(c, s):
    f = c["f"]
    names = ["X", "Wgu", "Wd"] + (["bgu", "bd"] if c["bias"] else [])
    a = {n: s[n].double().requires_grad_(c["train"]) for n in names}
    GU = a["X"] @ a["Wgu"]
    if c["bias"]:
        GU = GU + a["bgu"]
    G, U = GU[:, :f], GU[:, f:]
    if c["act"] == "silu":
        A = G * torch.sigmoid(G)
    else:
        A = G * torch.special.ndtr(G)
    Z = (A * U) @ a["Wd"]
    if c["bias"]:
        Z = Z + a["bd"]
    out = {"Z": Z.detach()}
    if c["train"]:
        gs = dict(zip(names, torch.autograd.grad(Z, [a[n] for n in names], s["dZ"].double())))
        out.update({"d" + n: gs[n] for n in ["X", "Wgu", "Wd"] + (["bgu", "bd"] if c["bias"] else [])})
    return out


# --------------------------------------------------------------------- work
def _visible_pairs(sq, sk, window, sinks):
    """Visible (query, key) pairs of one head."""
    n = 0
    for r in range(sq):
        p = r + sk - sq
        w = min(p + 1, window)
        n += w + min(sinks, p + 1 - w)
    return n


def work(case):
    """Inputs read once, outputs written once; the products and sums of the formulas."""
    op = case["op"]
    if op == "rope":
        es = 4 if case["dtype"] == "fp32" else 2
        n = case["M"] * (case["heads"] + case["kv_heads"]) * case["d"]
        side = 4 * case["M"] + 4 * case["d_rot"]
        if case["train"]:  # x, y; x again, dy, dx
            return {"bytes": 5 * n * es + 2 * side + 6 * case["d"] * es, "flops": 28 * n}
        return {"bytes": 2 * n * es + side + 2 * case["d"] * es, "flops": 9 * n}
    if op == "window":
        b, sq, sk, d = case["b"], case["sq"], case["sk"], case["d"]
        nq, nk = b * sq * case["heads"] * d * 2, b * sk * case["kv_heads"] * d * 2
        lse = 4 * b * case["heads"] * sq
        pairs = _visible_pairs(sq, sk, case["window"], case["sinks"]) * b * case["heads"]
        if case["train"]:  # q, k, v, o; again with do, dq, dk, dv
            return {"bytes": 6 * nq + 6 * nk + 2 * lse, "flops": 14 * d * pairs}
        return {"bytes": 2 * nq + 2 * nk + lse, "flops": 4 * d * pairs}
    if op == "decode":
        b, cap, d = case["b"], case["cap"], case["d"]
        mean = 0.75 * cap if b > 1 else cap - cap / 128.0
        keys = b * min(mean, case["window"] + case["sinks"])
        io = b * case["heads"] * (4 * d + 4) + 4 * b
        return {"bytes": keys * case["kv_heads"] * d * 4 + io,
                "flops": 4 * d * keys * case["heads"]}
    M, h, f = case["M"], case["h"], case["f"]
    weights, x = 2 * 3 * h * f, 2 * M * h
    if case["train"]:
        return {"bytes": 3 * weights + 5 * x, "flops": 18 * M * h * f}
    return {"bytes": weights + 2 * x, "flops": 6 * M * h * f}
