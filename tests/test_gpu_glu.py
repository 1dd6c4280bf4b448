"""The gated feed-forward block against fp64 (GPU).

Tolerances follow the bf16 roundings (hs = 2^-8, half a step): H is rounded
(up to 8 tokens its rest follows as a second term), so Z may be off by hs (|H| |Wd|) + hs |Z|.  In the backward G and U are rounded
to fp16 (2^-11 of the value, half a step of 2^-24 below 2^-14), [dG | dU] and
H to bf16: with their errors eG, eU, dG = dH U act'(G) may be off by |dH| (|act'| eU + |U| |act''| eG) and hs of itself (|act''| <= 1), dU and H
likewise (|act'| <= 1.13), and the products follow by linearity.  fp32 sums
and the activations (erf to 1.5e-7, exp2 and reciprocal to about 2^-21) stay
below 2^-14 of the same magnitudes.  Those are worst cases; random roundings
average out: a gradient meets two bf16 roundings (1.7e-3 each) and the fp16
ones of G and U (2.1e-4), 2.4e-3 together, and the norms are held to 1.25 times
that (the norm of n errors scatters about it by 1 / sqrt(2 n); four of those).
"""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu

pytestmark = pytest.mark.gpu
HS, F32 = 2.0 ** -8, 2.0 ** -14
NORMWISE = 3e-3
ACTS = {"silu": L.TP_ACT_SILU, "gelu": L.TP_ACT_GELU}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


def make(M, h, f, bias, seed=0, std=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()
    return dict(X=rn(M, h), Wgu=rn(h, 2 * f, std=std or h ** -0.5), Wd=rn(f, h, std=f ** -0.5),
                bgu=rn(2 * f, std=0.3) if bias else None, bd=rn(h, std=0.3) if bias else None,
                dZ=rn(M, h))


def act(x, kind):
    if kind == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    cdf = torch.special.ndtr(x)
    return x * cdf, cdf + x * torch.exp(-x * x / 2) * 0.3989422804014327


def reference(d, kind):
    X, Wgu, Wd, dZ = (d[n].double() for n in ("X", "Wgu", "Wd", "dZ"))
    f = Wd.shape[0]
    GU, mGU = X @ Wgu, X.abs() @ Wgu.abs()
    if d["bgu"] is not None:
        GU, mGU = GU + d["bgu"].double(), mGU + d["bgu"].double().abs()
    G, U = GU[:, :f], GU[:, f:]
    eGU = 2.0 ** -11 * GU.abs() + 2.0 ** -25 + F32 * mGU
    eG, eU = eGU[:, :f], eGU[:, f:]
    a, da = act(G, kind)
    H = a * U
    sG, sU = F32 * mGU[:, :f], F32 * mGU[:, f:]  # before rounding: what the forward's H sees
    eHf = HS * H.abs() + 1.13 * sG * U.abs() + a.abs() * sU
    Z = H @ Wd
    eZ = eHf @ Wd.abs() + F32 * (H.abs() @ Wd.abs())
    if d["bd"] is not None:
        Z, eZ = Z + d["bd"].double(), eZ + F32 * d["bd"].double().abs()
    ref, tol = {"Z": Z, "GU": GU}, {"Z": eZ + HS * Z.abs(), "GU": eGU}
    dH, mdH = dZ @ Wd.t(), F32 * (dZ.abs() @ Wd.abs().t())
    dG, dU = dH * U * da, dH * a
    edG = HS * dG.abs() + dH.abs() * (da.abs() * eU + U.abs() * eG) + mdH * (U * da).abs()
    edU = HS * dU.abs() + dH.abs() * 1.13 * eG + mdH * a.abs()
    eH = HS * H.abs() + 1.13 * eG * U.abs() + a.abs() * eU
    dGU, eD = torch.cat([dG, dU], 1), torch.cat([edG, edU], 1)
    out = {"dX": (dGU @ Wgu.t(), eD @ Wgu.abs().t(), dGU.abs() @ Wgu.abs().t()),
           "dWgu": (X.t() @ dGU, X.abs().t() @ eD, X.abs().t() @ dGU.abs()),
           "dWd": (H.t() @ dZ, eH.t() @ dZ.abs(), H.abs().t() @ dZ.abs()),
           "dbgu": (dGU.sum(0), eD.sum(0), dGU.abs().sum(0)),
           "dbd": (dZ.sum(0), 0 * dZ.sum(0), dZ.abs().sum(0))}
    for n, (r, e, m) in out.items():
        ref[n], tol[n] = r, e + F32 * m + HS * r.abs()
    return ref, tol


def run(d, t, kind, save=True, backward=True):
    M, h = d["X"].shape
    f = d["Wd"].shape[0]
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    out = {"Z": nan(M, h)}
    GU = nan(M, 2 * f).half() if save else None
    ws = L.workspace(L.TP_OP_GLU_FWD, M, h, f, 0, t, L.TP_BF16)
    L.tp_glu_fwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], d["bd"], out["Z"], GU, t, ACTS[kind], ws)
    if save:
        out["GU"] = GU
    if backward:
        out.update(dX=nan(M, h), dWgu=nan(h, 2 * f), dWd=nan(f, h))
        if d["bgu"] is not None:
            out.update(dbgu=nan(2 * f), dbd=nan(h))
        wsb = L.workspace(L.TP_OP_GLU_BWD, M, h, f, 0, t, L.TP_BF16)
        L.tp_glu_bwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], GU, d["dZ"], out["dX"], out["dWgu"],
                     out.get("dbgu"), out["dWd"], out.get("dbd"), t, ACTS[kind], wsb)
    return out


def compare(out, ref, tol):
    for n, got in out.items():
        g, r = got.double(), ref[n]
        bad = ((g - r).abs() - tol[n]).max().item()
        assert bad <= 0, f"{n}: {bad:.3e} over the bound"
        nw = ((g - r).norm() / r.norm().clamp_min(1e-30)).item()
        assert nw <= NORMWISE * (1 + 4 / (2 * r.numel()) ** 0.5), f"{n}: normwise {nw:.3e}"


CASES = [  # M, h, f, t, act, bias
    (1, 8, 8, 1, "silu", False),
    (1, 1024, 2816, 1, "gelu", True),
    (13, 520, 1000, 5, "silu", True),       # f / t not a multiple of 8 columns of 64
    (16, 2048, 264, 3, "gelu", False),
    (17, 136, 72, 1, "silu", True),
    (33, 1000, 1032, 1, "gelu", True),
    (64, 512, 4096, 8, "silu", False),
    (65, 512, 1024, 2, "silu", True),       # the tensor-core kernels from here on
    (100, 2056, 520, 1, "gelu", False),     # tiles cut along K
    (129, 264, 1416, 3, "silu", True),      # ragged rows, columns and shards
    (300, 768, 2048, 4, "gelu", True),
    (515, 1024, 2736, 1, "silu", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "M%dh%df%dt%d%s" % c[:5])
def test_forward_and_backward(case):
    M, h, f, t, kind, bias = case
    d = make(M, h, f, bias)
    ref, tol = reference(d, kind)
    compare(run(d, t, kind), ref, tol)


@pytest.mark.parametrize("M,h,f", [(1, 64, 96), (3, 200, 1000), (8, 1024, 2816)])
def test_the_fewest_tokens_round_once(M, h, f):
    """H crosses in two bf16 terms (2^-16 of it stays), so Z is off by its own
    rounding and the fp32 terms of `reference` alone."""
    d = make(M, h, f, True, seed=7)
    Z = run(d, 1, "silu", save=False, backward=False)["Z"].double()
    ref, tol = reference(d, "silu")
    G, U = ref["GU"][:, :f], ref["GU"][:, f:]
    cut = (HS - 2.0 ** -16) * ((act(G, "silu")[0] * U).abs() @ d["Wd"].double().abs())
    bad = ((Z - ref["Z"]).abs() - (tol["Z"] - cut)).max().item()
    assert bad <= 0, f"{bad:.3e} over the bound"


@pytest.mark.parametrize("tile", ["128", "192", "256", "pair"])
def test_every_tile_kind(tile, monkeypatch):
    monkeypatch.setenv("TP_GEMM_TILE", tile)
    d = make(290, 200, 712, True, 1)
    ref, tol = reference(d, "silu")
    compare(run(d, 1, "silu"), ref, tol)


def test_recomputed_preactivation_equals_the_saved_one():
    for M, t in ((40, 1), (200, 2)):
        d = make(M, 256, 640, True, 2)
        a, b = run(d, t, "gelu"), run(d, t, "gelu", save=False)
        ref, tol = reference(d, "gelu")
        compare(b, ref, tol)
        assert torch.equal(a["Z"], b["Z"])


def test_shard_counts_agree():
    for M in (24, 260):
        d = make(M, 384, 1024, False, 3)
        one = run(d, 1, "silu")
        for t in (2, 8, 64):
            other = run(d, t, "silu")
            ref, tol = reference(d, "silu")
            compare(other, ref, tol)
            assert torch.equal(one["Z"], other["Z"]) or M > 64


def test_preactivations_beyond_fp16_are_saturated_and_flagged():
    """[G | U] is kept in fp16: what does not fit is saturated there and
    reported; Z comes from the unrounded values."""
    for M in (5, 90):
        d = make(M, 64, 128, False, 12)
        d["Wgu"][:, 0] = 0
        d["Wgu"][0, 0], d["X"][:, 0] = 512.0, 512.0  # G[:, 0] = 2^18
        f = 128
        ws = L.workspace(L.TP_OP_GLU_FWD, M, 64, f, 0, 1, L.TP_BF16)
        Z = torch.empty_like(d["X"])
        GU = torch.empty(M, 2 * f, dtype=torch.float16, device="cuda")
        L.tp_glu_fwd(d["X"], d["Wgu"], None, d["Wd"], None, Z, None, 1, 0, ws)
        L.tp_device_status()  # nothing kept, nothing to report
        Z2 = torch.empty_like(Z)
        L.tp_glu_fwd(d["X"], d["Wgu"], None, d["Wd"], None, Z2, GU, 1, 0, ws)
        assert (GU[:, 0] == 65504).all() and torch.equal(Z, Z2)
        with pytest.raises(L.TPError) as e:
            L.tp_device_status()
        assert e.value.status == L.TP_ERR_KERNEL and "fp16" in str(e.value)


def test_large_and_special_preactivations():
    """Gates far out: sigmoid and its exponential saturate, nothing is NaN; a
    NaN token stays in its row."""
    for M in (8, 100):
        d = make(M, 64, 128, False, 4, std=40.0)
        assert (d["X"].double() @ d["Wgu"].double()).abs().max() < 65504
        ref, tol = reference(d, "silu")
        compare({"Z": run(d, 1, "silu", backward=False)["Z"]}, ref, tol)
        clean = run(d, 1, "silu", backward=False)["Z"]
        d["X"][3] = float("nan")
        Z = run(d, 1, "silu", backward=False)["Z"]
        keep = [i for i in range(M) if i != 3]
        assert torch.isnan(Z[3]).all() and torch.equal(Z[keep], clean[keep])


def test_exact_on_integers_whatever_the_path():
    """With gates of 64 (act(64) = 64 exactly) and small integers every sum is
    exact, so the streaming and the tensor-core kernels agree bit for bit."""
    h, f = 256, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randint(-1, 2, (80, h), generator=g, device="cuda").bfloat16()
    Wgu = torch.zeros(h, 2 * f, device="cuda")
    Wgu[:, f:] = torch.randint(-1, 2, (h, f), generator=g, device="cuda")
    bgu = torch.cat([torch.full((f,), 64.0, device="cuda"), torch.zeros(f, device="cuda")])
    Wd = torch.zeros(f, h, device="cuda")
    Wd[torch.arange(f), torch.arange(f) % h] = 1.0
    d = dict(X=X, Wgu=Wgu.bfloat16(), bgu=bgu.bfloat16(), Wd=Wd.bfloat16(), bd=None,
             dZ=torch.zeros_like(X))
    U = X.double() @ d["Wgu"][:, f:].double()
    want = (64 * U) @ d["Wd"].double()
    full = run(d, 1, "silu", backward=False)["Z"]
    assert torch.equal(full.double(), want.bfloat16().double())
    for M in (1, 5, 16, 30, 60):
        part = dict(d, X=X[:M].contiguous(), dZ=d["dZ"][:M])
        assert torch.equal(run(part, 1, "silu", backward=False)["Z"], full[:M])


def test_gradients_against_differences():
    d = make(70, 64, 96, True, 6)
    out = run(d, 1, "silu")

    def loss(p):
        GU = p["X"] @ p["Wgu"] + p["bgu"]
        Z = (act(GU[:, :96], "silu")[0] * GU[:, 96:]) @ p["Wd"] + p["bd"]
        return (Z * d["dZ"].double()).sum().item()

    p = {n: d[n].double() for n in ("X", "Wgu", "bgu", "Wd", "bd")}
    g = torch.Generator(device="cuda").manual_seed(7)
    for n in p:
        u = torch.randn(p[n].shape, generator=g, device="cuda", dtype=torch.float64)
        up, dn = (loss({**p, n: p[n] + e * u}) for e in (1e-5, -1e-5))
        got = out["d" + n].double()
        # independent errors of 5e-3 of each value at most, along a random direction
        assert abs((up - dn) / 2e-5 - (got * u).sum().item()) <= 5e-3 * (got * u).norm().item() * 4


def test_only_the_gradients_asked_for():
    d = make(130, 128, 256, True, 8)
    ref = run(d, 2, "gelu")
    f, h = 256, 128
    GU = ref["GU"]
    wsb = L.workspace(L.TP_OP_GLU_BWD, 130, h, f, 0, 2, L.TP_BF16)
    for bgu, bd in ((True, False), (False, True), (False, False)):
        dX, dWgu, dWd = (torch.empty_like(ref[n]) for n in ("dX", "dWgu", "dWd"))
        a = torch.empty_like(ref["dbgu"]) if bgu else None
        b = torch.empty_like(ref["dbd"]) if bd else None
        L.tp_glu_bwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], GU, d["dZ"], dX, dWgu, a, dWd, b, 2,
                     L.TP_ACT_GELU, wsb)
        for n, v in (("dX", dX), ("dWgu", dWgu), ("dWd", dWd), ("dbgu", a), ("dbd", b)):
            assert v is None or torch.equal(v, ref[n]), n


@pytest.mark.parametrize("M", [7, 50, 200])
def test_graph_replay_on_a_side_stream(M):
    d = make(M, 1024, 1408, True, 9)
    h, f = 1024, 1408
    ref = run(d, 1, "silu")
    out = {n: torch.empty_like(v) for n, v in ref.items()}
    ws = L.workspace(L.TP_OP_GLU_FWD, M, h, f, 0, 1, L.TP_BF16)
    wsb = L.workspace(L.TP_OP_GLU_BWD, M, h, f, 0, 1, L.TP_BF16)

    def step():
        for _ in range(2):  # two calls in a row share the workspace
            L.tp_glu_fwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], d["bd"], out["Z"], out["GU"], 1, 0, ws)
        L.tp_glu_bwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], out["GU"], d["dZ"], out["dX"],
                     out["dWgu"], out["dbgu"], out["dWd"], out["dbd"], 1, 0, wsb)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                step()
    for g in graphs + graphs:
        for v in out.values():
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], ref[n]) for n in ref)


def test_workspace_without_the_optional_part():
    d = make(100, 2056, 520, False, 10)
    want = run(d, 1, "silu", save=False, backward=False)["Z"]
    ws = torch.empty(100 * 520 * 2 + 512, dtype=torch.uint8, device="cuda")
    Z = torch.empty_like(want)
    L.tp_glu_fwd(d["X"], d["Wgu"], None, d["Wd"], None, Z, None, 1, 0, ws)
    ref, tol = reference(d, "silu")
    compare({"Z": Z}, ref, tol)


@pytest.mark.parametrize("M", [1, 33, 130])
def test_a_backward_stays_inside_its_workspace(M):
    """Rows past M have no place in the bias gradients' partial sums: bytes
    behind the smallest workspace the calls take stay as they were, and other
    parts of it intact (the results are right)."""
    h, f = 256, 4096
    d = make(M, h, f, True, 13)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tail = (4096 + sms * 128 * 256 * 4 + 255) // 256 * 256 + 256  # the optional part
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    GU = torch.empty(M, 2 * f, dtype=torch.float16, device="cuda")
    L.tp_glu_fwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], d["bd"], e(M, h), GU, 1, 0,
                 L.workspace(L.TP_OP_GLU_FWD, M, h, f, 0, 1, L.TP_BF16))
    need = L.tp_workspace_size(L.TP_OP_GLU_BWD, M, h, f, 0, 1, L.TP_BF16) - tail
    buf = torch.full((need + (8 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    out = dict(dX=e(M, h), dWgu=e(h, 2 * f), dWd=e(f, h), dbgu=e(2 * f), dbd=e(h))
    L.tp_glu_bwd(d["X"], d["Wgu"], d["bgu"], d["Wd"], GU, d["dZ"], out["dX"], out["dWgu"],
                 out["dbgu"], out["dWd"], out["dbd"], 1, 0, buf[:need])
    assert (buf[need:] == 0x5a).all()
    ref, tol = reference(d, "silu")
    compare(out, ref, tol)
    # the same for the plain MLP's backward
    A, B, Y, bA = d["Wgu"][:, :f].contiguous(), d["Wd"], e(M, f), d["bgu"][:f].contiguous()
    L.tp_mlp_fwd(d["X"], A, bA, B, d["bd"], e(M, h), Y, 1,
                 L.workspace(L.TP_OP_MLP_FWD, M, h, f, 0, 1, L.TP_BF16))
    need = L.tp_workspace_size(L.TP_OP_MLP_BWD, M, h, f, 0, 1, L.TP_BF16) - tail
    buf = torch.full((need + (8 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    dbA = e(f)
    L.tp_mlp_bwd(d["X"], A, bA, B, Y, d["dZ"], e(M, h), e(h, f), dbA, e(f, h), e(h), 1, buf[:need])
    assert (buf[need:] == 0x5a).all()
    Yd = Y.double()
    cdf = torch.special.ndtr(Yd)
    dY = (d["dZ"].double() @ B.double().t()) * (cdf + Yd * torch.exp(-Yd * Yd / 2) * 0.3989422804014327)
    assert ((dbA.double() - dY.sum(0)).norm() / dY.sum(0).norm()).item() <= 5e-3


def test_binding_refuses_mismatched_tensors():
    d = make(4, 64, 128, True, 11)
    Z, ws = torch.empty_like(d["X"]), L.workspace(L.TP_OP_GLU_FWD, 4, 64, 128, 0, 1, L.TP_BF16)
    ok = [d["X"], d["Wgu"], d["bgu"], d["Wd"], d["bd"], Z, None, 1, 0, ws]
    L.tp_glu_fwd(*ok)
    for i, bad in ((0, d["X"].float()), (1, d["Wgu"][:, :128]), (2, d["bgu"][:128]),
                   (2, d["bgu"].float()), (3, d["Wd"].t()), (5, Z[:3]), (6, Z), (0, d["X"].cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            L.tp_glu_fwd(*args)
