"""Query/key norm + rotary against fp64 (GPU).

Tolerance per value: half a step of the storage type relative to the result,
plus the fp32 arithmetic: every intermediate (x r g, the two terms of a
rotated value, the two terms of dx) carries at most about 16 roundings of
2^-24 relative to its own magnitude (8 + 5 additions in a row sum counted on
the statistic, rsqrt's 2 ulp, the products), so 32 * 2^-24 of the sum of the
terms' magnitudes bounds it.
"""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def rot(x, pos, fr, d_rot, il, sign):
    """x [M, H, d] rotated, and the sum of its terms' magnitudes."""
    y, mag = x.clone(), x.abs()
    if d_rot:
        # the angle reduced by whole turns the long way: far positions in fp64
        t = sign * (pos.double()[:, None] * fr)[:, None, :]
        i = torch.arange(d_rot // 2, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if il else (i, i + d_rot // 2)
        a, b, c, s = x[..., ia], x[..., ib], torch.cos(t), torch.sin(t)
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def reference(x, g, pos, fr, d, d_rot, norm, il, eps, dy=None):
    M = x.shape[0]
    X = x.double().reshape(M, -1, d)
    G = torch.ones(d, dtype=torch.float64, device=x.device) if g is None or not norm else g.double()
    r = (X.square().mean(-1, keepdim=True) + eps).rsqrt() if norm else torch.ones_like(X[..., :1])
    out = {}
    y, mag = rot(X * r * G, pos, fr, d_rot, il, 1.0)
    out["y"], out["y_mag"] = y.reshape(M, -1), mag.reshape(M, -1)
    if dy is not None:
        dz, dmag = rot(dy.double().reshape(M, -1, d), pos, fr, d_rot, il, -1.0)
        if norm:
            k = r ** 3 * (dz * G * X).mean(-1, keepdim=True)
            kmag = r ** 3 * (dmag * G.abs() * X.abs()).mean(-1, keepdim=True)
            dx, dxm = r * dz * G - X * k, r * dmag * G.abs() + X.abs() * kmag
            out["dg"], out["dg_mag"] = (dz * X * r).sum((0, 1)), (dmag * X.abs() * r).sum((0, 1))
        else:
            dx, dxm = dz, dmag
        out["dx"], out["dx_mag"] = dx.reshape(M, -1), dxm.reshape(M, -1)
    return out


def close(got, ref, mag, dt, what, k=32):
    err = (got.double() - ref).abs()
    tol = half_step(dt) * ref.abs() + k * U32 * mag
    if dt == torch.float16:
        tol = tol + 2.0 ** -25  # half a subnormal step
    bad = (err - tol).max().item()
    assert bad <= 0, f"{what}: {bad:.3e} over, worst error {err.max().item():.3e}"


CASES = [  # M, heads, kv_heads, d, d_rot, dtype, interleaved, max position
    (1, 1, 1, 8, 0, torch.bfloat16, False, 1),
    (1, 32, 8, 128, 128, torch.bfloat16, False, 1 << 20),
    (3, 5, 0, 64, 64, torch.float16, False, 4096),
    (17, 7, 3, 80, 32, torch.bfloat16, False, 4096),
    (130, 3, 1, 96, 96, torch.float32, True, 4096),
    (513, 4, 2, 256, 256, torch.bfloat16, True, 1 << 30),
    (1201, 2, 2, 24, 16, torch.float16, True, 100),
    (5000, 9, 9, 136, 80, torch.float32, False, 1 << 16),
    (9001, 2, 1, 128, 128, torch.bfloat16, False, 9001),
]


def make(case, seed=0):
    M, H, Hk, d, dr, dt, il, mp = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    qkv = rn(M, (H + 2 * Hk) * d).to(dt)
    t = dict(Q=qkv[:, :H * d], K=qkv[:, H * d:(H + Hk) * d] if Hk else None,
             gq=(1 + 0.2 * rn(d)).to(dt), gk=(1 + 0.2 * rn(d)).to(dt),
             pos=torch.randint(-mp, mp, (M,), generator=g, device="cuda", dtype=torch.int32),
             fr=torch.pow(10000.0, -torch.arange(dr // 2, device="cuda", dtype=torch.float64)
                          * 2 / dr) if dr else None,
             dQo=rn(M, H * d).to(dt), dKo=rn(M, Hk * d).to(dt) if Hk else None)
    return t


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"M{c[0]}h{c[1]}k{c[2]}d{c[3]}r{c[4]}")
def test_forward_and_backward(case, norm):
    M, H, Hk, d, dr, dt, il, _ = case
    t = make(case)
    new = lambda x: None if x is None else torch.full_like(
        x, float("nan"), memory_format=torch.contiguous_format)
    Qo, Ko, dQ, dK = new(t["Q"]), new(t["K"]), new(t["Q"]), new(t["K"])
    dgq, dgk = new(t["gq"]), new(t["gk"])
    L.tp_qk_norm_rope_fwd(t["Q"], t["K"], t["gq"], t["gk"], t["pos"], t["fr"], Qo, Ko, d, norm, il,
                          1e-6)
    L.tp_qk_norm_rope_bwd(t["Q"], t["K"], t["gq"], t["gk"], t["pos"], t["fr"], t["dQo"], t["dKo"],
                          dQ, dK, dgq, dgk, d, L.qk_norm_rope_workspace(M, d), norm, il, 1e-6)
    for n, x, g, dy, y, dx, dg in (("q", t["Q"], t["gq"], t["dQo"], Qo, dQ, dgq),
                                   ("k", t["K"], t["gk"], t["dKo"], Ko, dK, dgk)):
        if x is None:
            continue
        ref = reference(x, g, t["pos"], t["fr"], d, dr, norm, il, 1e-6, dy)
        close(y, ref["y"], ref["y_mag"], dt, f"{n} forward")
        close(dx, ref["dx"], ref["dx_mag"], dt, f"d{n}")
        if norm:
            # chains of at most: a thread's rows, 2 shuffles, 8 warps, 32 phases, blocks / 32
            rows = M * x.shape[1] // d
            k = 32 + 2 + 8 + 32 + 20 + rows // 8
            close(dg, ref["dg"], ref["dg_mag"], dt, f"dg{n}", k if rows < 512 else 128)
        else:
            assert torch.isnan(dg).all()  # not asked for: left as it was


def test_gradients_against_differences():
    """dx and dg of sum(y * w) against central differences of the fp32 forward."""
    case = (2, 2, 1, 32, 16, torch.float32, False, 50)
    t = make(case, 5)
    d = 32
    Q, gq, w = t["Q"].contiguous(), t["gq"].clone(), t["dQo"]
    dQ, dg = torch.empty_like(Q), torch.empty_like(gq)
    L.tp_qk_norm_rope_bwd(Q, None, gq, None, t["pos"], t["fr"], w, None, dQ, None, dg, None, d,
                          L.qk_norm_rope_workspace(2, d))

    def loss(q, g):
        y = torch.empty_like(q)
        L.tp_qk_norm_rope_fwd(q, None, g, None, t["pos"], t["fr"], y, None, d)
        return (y.double() * w.double()).sum().item()

    # a step of 2^-6: truncation h^2 f''' / 6 ~ 1e-4 of values of order one, rounding
    # 64 terms * 2^-24 / 2^-6 ~ 2.5e-4; together below 5e-3
    h = 2.0 ** -6
    for x, gx, other in ((Q, dQ, "q"), (gq, dg, "g")):
        flat = x.view(-1)
        for i in range(0, flat.numel(), 7):
            v = flat[i].item()
            flat[i] = v + h
            up = loss(Q, gq)
            flat[i] = v - h
            dn = loss(Q, gq)
            flat[i] = v
            assert abs((up - dn) / (2 * h) - gx.view(-1)[i].item()) < 5e-3, (other, i)


def test_in_place_equals_out_of_place_and_leaves_the_rest():
    case = (70, 6, 2, 64, 64, torch.bfloat16, False, 1000)
    t = make(case, 1)
    H, Hk, d = 6, 2, 64
    Qo, Ko = torch.empty(70, H * d, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(70, Hk * d, dtype=torch.bfloat16, device="cuda")
    L.tp_qk_norm_rope_fwd(t["Q"], t["K"], t["gq"], t["gk"], t["pos"], t["fr"], Qo, Ko, d)
    buf = t["Q"]._base if t["Q"]._base is not None else t["Q"]
    V = buf[:, (H + Hk) * d:].clone()
    L.tp_qk_norm_rope_fwd(t["Q"], t["K"], t["gq"], t["gk"], t["pos"], t["fr"], t["Q"], t["K"], d)
    assert torch.equal(t["Q"], Qo) and torch.equal(t["K"], Ko)
    assert torch.equal(buf[:, (H + Hk) * d:], V)
    dQ, dK = torch.empty_like(Qo), torch.empty_like(Ko)
    args = (Qo, Ko, t["gq"], t["gk"], t["pos"], t["fr"])
    L.tp_qk_norm_rope_bwd(*args, t["dQo"], t["dKo"], dQ, dK, None, None, d, None)
    L.tp_qk_norm_rope_bwd(*args, t["dQo"], t["dKo"], t["dQo"], t["dKo"], None, None, d, None)
    assert torch.equal(dQ, t["dQo"]) and torch.equal(dK, t["dKo"])


def test_non_finite_rows_stay_in_their_rows_and_the_gradient_repeats():
    case = (40, 4, 1, 128, 128, torch.bfloat16, False, 1000)
    t = make(case, 2)
    d, M = 128, 40
    ws = L.qk_norm_rope_workspace(M, d)

    def both(K):
        Ko, dK, dg = torch.empty(M, d, dtype=K.dtype, device="cuda"), \
            torch.empty(M, d, dtype=K.dtype, device="cuda"), torch.empty_like(t["gk"])
        L.tp_qk_norm_rope_fwd(K, None, t["gk"], None, t["pos"], t["fr"], Ko, None, d)
        L.tp_qk_norm_rope_bwd(K, None, t["gk"], None, t["pos"], t["fr"], t["dKo"], None, dK, None,
                              dg, None, d, ws)
        return Ko, dK, dg

    a, b = both(t["K"]), both(t["K"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    bad = t["K"].clone()
    bad[7, 3], bad[8, 5] = float("inf"), float("nan")
    c = both(bad)
    keep = [i for i in range(M) if i not in (7, 8)]
    assert torch.equal(c[0][keep], a[0][keep]) and torch.equal(c[1][keep], a[1][keep])


def test_streams_and_graph_replay():
    case = (256, 8, 2, 128, 128, torch.bfloat16, False, 4096)
    t = make(case, 3)
    d = 128
    outs = [torch.empty_like(t[n], memory_format=torch.contiguous_format) for n in ("Q", "K")]
    grads = [torch.empty_like(t[n], memory_format=torch.contiguous_format) for n in ("Q", "K")]
    dgs = [torch.empty_like(t["gq"]), torch.empty_like(t["gk"])]
    ws = L.qk_norm_rope_workspace(256, d)

    def step():
        L.tp_qk_norm_rope_fwd(t["Q"], t["K"], t["gq"], t["gk"], t["pos"], t["fr"], *outs, d)
        L.tp_qk_norm_rope_bwd(t["Q"], t["K"], t["gq"], t["gk"], t["pos"], t["fr"], t["dQo"],
                              t["dKo"], *grads, *dgs, d, ws)

    step()
    torch.cuda.synchronize()
    ref = [x.clone() for x in outs + grads + dgs]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    for _ in range(2):
        for x in outs + grads + dgs:
            x.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs + grads + dgs, ref))


def test_no_tokens():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    fr = torch.ones(32, dtype=torch.float64, device="cuda")
    dg = torch.full_like(g, 7.0)
    L.tp_qk_norm_rope_fwd(e, e, g, g, pos, fr, e.clone(), e.clone(), 64)
    L.tp_qk_norm_rope_bwd(e, None, g, None, pos, fr, e, None, e.clone(), None, dg, None, 64, None)
    assert (dg == 0).all()


def test_binding_refuses_mismatched_tensors():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    fr = torch.ones(32, dtype=torch.float64, device="cuda")
    ok = (x, None, g, None, pos, fr, x.clone(), None, 64)
    L.tp_qk_norm_rope_fwd(*ok)
    for i, bad in ((0, x.float()), (2, g.float()), (4, pos.long()), (4, pos[:3]), (5, fr.float()),
                   (6, x[:3]), (6, x.half()), (6, x.t()), (0, x.cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            L.tp_qk_norm_rope_fwd(*args)
