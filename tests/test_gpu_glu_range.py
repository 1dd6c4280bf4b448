"""The gated block's backward over the range of its type (GPU).

bf16 tokens and weights may be far from one; Z is right there, and with the
pre-activations recomputed so are the gradients.  [G | U] then crosses in two
bf16 terms, off by 2^-17 of the value (with the fp32 sums, 2^-14 of the
products' magnitudes); [dG | dU] and H are rounded to bf16 (2^-8), so by
linearity, with act' at most 1.13 and act'' at most 1 in magnitude,
  |d dG| <= hs |dG| + |dH| (|act'| eU + |U| eG),  |d dU| <= hs |dU| + |dH| 1.13 eG,
  |d H| <= hs |H| + 1.13 eG |U| + |act| eU,
and the gradients take those through the products and round once more.  The
bounds are relative to the results (nothing absolute but bf16's smallest
normal number, which stays far below), so they hold at any scale.  Two bf16
roundings of 1.7e-3 give 2.4e-3 together; the norms are held to 1.25 times that.
"""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu
from tests.test_gpu_glu import ACTS, F32, HS, NORMWISE, act, compare, make, run
from tests.test_gpu_glu import reference as kept_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


def reference(d, kind):
    """The gradients and their bounds, with a recomputed [G | U]."""
    X, Wgu, Wd, dZ = (d[n].double() for n in ("X", "Wgu", "Wd", "dZ"))
    f = Wd.shape[0]
    b = torch.zeros(2 * f, dtype=torch.float64, device="cuda") if d["bgu"] is None \
        else d["bgu"].double()
    GU, mGU = X @ Wgu + b, X.abs() @ Wgu.abs() + b.abs()
    eGU = 2.0 ** -17 * GU.abs() + F32 * mGU
    (G, U), (eG, eU) = GU.split(f, 1), eGU.split(f, 1)
    a, da = act(G, kind)
    dH, mdH = dZ @ Wd.t(), F32 * (dZ.abs() @ Wd.abs().t())
    H, dG, dU = a * U, dH * U * da, dH * a
    eH = HS * H.abs() + 1.13 * eG * U.abs() + a.abs() * eU
    edG = HS * dG.abs() + dH.abs() * (da.abs() * eU + U.abs() * eG) + mdH * (U * da).abs()
    edU = HS * dU.abs() + dH.abs() * 1.13 * eG + mdH * a.abs()
    g, e = torch.cat([dG, dU], 1), torch.cat([edG, edU], 1)
    out = {"dX": (g @ Wgu.t(), (e + F32 * g.abs()) @ Wgu.abs().t()),
           "dWgu": (X.t() @ g, X.abs().t() @ (e + F32 * g.abs())),
           "dWd": (H.t() @ dZ, (eH + F32 * H.abs()).t() @ dZ.abs()),
           "dbgu": (g.sum(0), (e + F32 * g.abs()).sum(0))}
    return {n: (r, t + HS * r.abs() + 2.0 ** -126) for n, (r, t) in out.items()}, (G, U)


def check(out, ref):
    for n, (r, t) in ref.items():
        if n not in out:
            continue
        err = (out[n].double() - r).abs()
        assert torch.isfinite(out[n]).all(), n
        nw = (err.norm() / r.norm()).item()
        assert nw <= NORMWISE * (1 + 4 / (2 * r.numel()) ** 0.5), f"{n}: normwise {nw:.3e}"
        assert (err - t).max().item() <= 0, f"{n}: {(err - t).max().item():.3e} over the bound"


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M,h,f,t", [(5, 128, 264, 1), (90, 520, 1032, 3), (300, 256, 512, 2)])
@pytest.mark.parametrize("scale", [1e-9, 1e-6, 1.0, 1e4, 1e8])
def test_recomputed_gradients_over_the_types_range(M, h, f, t, kind, scale):
    d = make(M, h, f, False, seed=21)
    d["X"] *= scale
    check(run(d, t, kind, save=False), reference(d, kind)[0])


@pytest.mark.parametrize("up", [1e-8, 1e6])
def test_recomputed_gradients_with_gates_of_order_one(up):
    """The up projection far from one, its bias too; the gates are not."""
    M, h, f = 140, 256, 512
    d = make(M, h, f, True, seed=22)
    d["Wgu"][:, f:] *= up
    d["bgu"][f:] *= up
    d["dZ"] *= 0.01
    ref, (G, U) = reference(d, "silu")
    assert U.abs().max() < 2.0 ** -24 or U.abs().max() > 65504
    check(run(d, 1, "silu", save=False), ref)


@pytest.mark.parametrize("tile", ["128", "192", "256", "pair"])
def test_every_tile_kind_recomputes(tile, monkeypatch):
    monkeypatch.setenv("TP_GEMM_TILE", tile)
    d = make(290, 200, 712, True, 23)
    d["X"] *= 1e6
    check(run(d, 1, "gelu", save=False), reference(d, "gelu")[0])


def test_kept_preactivations_need_no_room_for_recomputed_ones():
    """With GUsave a workspace without the 8 M f bytes of the recomputation is
    enough, and nothing behind it is written."""
    M, h, f = 130, 256, 1024
    d = make(M, h, f, True, 24)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tail = (4096 + sms * 128 * 256 * 4 + 255) // 256 * 256 + 256  # the optional part
    need = L.tp_workspace_size(L.TP_OP_GLU_BWD, M, h, f, 0, 1, L.TP_BF16) - tail - 8 * M * f
    ref = run(d, 1, "silu")
    buf = torch.full((need + (8 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    out = {n: torch.empty_like(ref[n]) for n in ("dX", "dWgu", "dbgu", "dWd", "dbd")}
    args = (d["X"], d["Wgu"], d["bgu"], d["Wd"])
    grads = (d["dZ"], out["dX"], out["dWgu"], out["dbgu"], out["dWd"], out["dbd"], 1, ACTS["silu"])
    L.tp_glu_bwd(*args, ref["GU"], *grads, buf[:need])
    assert (buf[need:] == 0x5a).all()
    compare(out, *kept_reference(d, "silu"))
    with pytest.raises(L.TPError) as e:
        L.tp_glu_bwd(*args, None, *grads, buf[:need])
    assert e.value.status == L.TP_ERR_WORKSPACE


@pytest.mark.parametrize("M", [1, 5, 20, 90, 260])
@pytest.mark.parametrize("h,f", [(64, 72), (128, 264)])
def test_kept_preactivations_too_low_for_fp16_are_flagged(M, h, f):
    """[G | U] is kept in fp16, whose steps stay 2^-24 below 2^-14: 32 neighbours
    that all lie below 2^-17 are reported, those of one token and of U alone too;
    zeros, which are exact, and values of order one are not."""
    d = make(M, h, f, False, seed=25)

    def status():
        run(d, 1, "silu", backward=False)
        try:
            L.tp_device_status()
        except L.TPError as e:
            assert e.status == L.TP_ERR_KERNEL and "2^-17" in str(e)
            return True
        return False

    assert not status()
    last = d["X"][M - 1].clone()
    d["X"][M - 1] = 0
    assert not status()
    d["X"][M - 1] = last * 2.0 ** -22  # G and U of that token about 2^-22
    assert status()
    run(d, 1, "silu", save=False, backward=False)
    L.tp_device_status()  # nothing kept, nothing to report
    d["X"][M - 1] = last
    d["Wgu"][:, f:] *= 2.0 ** -22  # U alone
    assert status()
    d["Wgu"][:, f:] = 0
    assert not status()
    d["Wgu"][:, f + 32:f + 64] = 2.0 ** -30  # one run of 32 columns
    assert status()


def test_both_sides_of_the_few_token_choices():
    """The same tokens in batches of 1, 8, 9, 16, 17, 32, 33 and 70: up to 8 H has
    two terms (2^-16 of it stays) and Z is off by its own rounding, beyond by H's
    too; among batches of up to 8, and of 9 to 32, a token's Z is the same."""
    h, f = 520, 1416
    d = make(70, h, f, True, seed=26)
    ref, tol = kept_reference(d, "silu")
    G, U = ref["GU"].split(f, 1)
    cut = (HS - 2.0 ** -16) * ((act(G, "silu")[0] * U).abs() @ d["Wd"].double().abs())
    Z = {}
    for M in (1, 8, 9, 16, 17, 32, 33, 70):
        part = dict(d, X=d["X"][:M].contiguous(), dZ=d["dZ"][:M].contiguous())
        Z[M] = run(part, 1, "silu", save=False, backward=False)["Z"]
        t = tol["Z"][:M] - (cut[:M] if M <= 8 else 0)
        over = ((Z[M].double() - ref["Z"][:M]).abs() - t).max().item()
        assert over <= 0, f"{M} tokens: {over:.3e} over the bound"
    assert torch.equal(Z[1], Z[8][:1])
    for M in (9, 16, 17):
        assert torch.equal(Z[M], Z[32][:M])


@pytest.mark.parametrize("M", [3, 13, 32])
def test_wide_blocks_take_more_than_one_round(M):
    """448 tiles of the up product, and 313 of the down, where 296 blocks run at once."""
    for h, f in ((128, 28672), (40000, 64)):
        d = make(M, h, f, False, seed=27)
        ref, tol = kept_reference(d, "silu")
        out = run(d, 1, "silu", backward=False)
        compare(out, ref, tol)


def test_the_profile_tells_streamed_products_from_the_tensor_core_gemm():
    h, f = 256, 512
    for M, kind in ((4, L.TP_KIND_GEMM_STREAM), (20, L.TP_KIND_GEMM_STREAM),
                    (40, L.TP_KIND_GEMM_TCGEN05)):
        d = make(M, h, f, False, seed=28)
        L.tp_profile_enable(True)
        try:
            run(d, 1, "silu", save=False, backward=False)
            records = L.tp_profile_records()
        finally:
            L.tp_profile_enable(False)
        assert [r["kind"] for r in records] == [L.KIND_NAMES[kind]] * 2
        assert [r["flops"] for r in records] == [4.0 * M * h * f, 2.0 * M * h * f]
        assert L.tp_profile_read(kind)["launches"] == 2
