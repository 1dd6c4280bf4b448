"""Single-token window attention on both sides of its choices (GPU): every type
and head dimension with few and with many outputs, groups of query heads that
leave room for the rests of P and groups that do not, sequences cut into slices
and sequences that are not.

P enters P V as the rounded value and the rounded rest, so with hs half a step
of the type O may be off by hs |O| (its own rounding), 2 hs^2 of P |V| (what two
terms leave) and 2^-13 of P |V| (products, sums and exponentials in fp32); an
fp16 rest below the smallest step adds up to 2^-25 |V| for each visible key (P is
at most 1 and the sum it is divided by at least 1).  None of that depends on what
else is in the batch.
"""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu
from tests.test_gpu_window import BF, F32, FP, close, half_step, rn, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


def reference(Q, K, V, lens, heads, kv, window, sinks):
    """O, LSE and their bounds in fp64."""
    b, d, dt, hs = K.shape[0], Q.shape[1] // heads, Q.dtype, half_step(Q.dtype)
    O = torch.zeros(b, heads, d, dtype=torch.float64, device="cuda")
    tO, lse = torch.zeros_like(O), torch.full((b, heads), float("-inf"), dtype=torch.float64,
                                              device="cuda")
    tl = torch.zeros_like(lse)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        seen = visible(1, n, window, sinks)[0]
        q = Q[i].double().reshape(kv, heads // kv, d)
        k, v = (x[i, :n][seen].double().reshape(-1, kv, d) for x in (K, V))
        s = torch.einsum("hgd,chd->hgc", q, k) * d ** -0.5
        P = torch.softmax(s, 2)
        O[i] = torch.einsum("hgc,chd->hgd", P, v).reshape(heads, d)
        mag = torch.einsum("hgc,chd->hgd", P, v.abs()).reshape(heads, d)
        tO[i] = hs * O[i].abs() + (F32 + 2 * hs * hs) * mag
        if dt == FP:
            tO[i] += 2.0 ** -25 * (1 + v.abs().sum(0).repeat_interleave(heads // kv, 0))
        lse[i] = torch.logsumexp(s, 2).reshape(heads)
        tl[i] = 2.0 ** -20 * (1 + torch.einsum("hgd,chd->hgc", q.abs(), k.abs()).amax(2).reshape(
            heads) * d ** -0.5)
    return O.reshape(b, -1), tO.reshape(b, -1), lse, tl


def call(Q, K, V, lens, heads, kv, window, sinks):
    b, cap, d = K.shape[0], K.shape[1], Q.shape[1] // heads
    O = torch.full((b, heads * d), float("nan"), dtype=Q.dtype, device="cuda")
    LSE = torch.full((b, heads), float("nan"), device="cuda")
    ws = L.window_attn_decode_workspace(b, cap, heads, kv, d, window, sinks)
    ws.fill_(0xff)
    L.tp_window_attn_decode(Q, K, V, torch.tensor(lens, dtype=torch.int32, device="cuda"), O, LSE,
                            heads, kv, window, sinks, ws)
    return O, LSE


def make(b, cap, heads, kv, d, dt, lens, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q, K, V = (rn(g, *s, dt=dt) for s in ((b, heads * d), (b, cap, kv * d), (b, cap, kv * d)))
    for i, n in enumerate(lens):  # whatever lies past a sequence's keys
        K[i, n:], V[i, n:] = float("nan"), float("nan")
    return Q, K, V


def lengths(b, cap):
    """Uneven ones, among them nothing, one key, and the whole cache."""
    return [(0, 1, cap, 17, cap // 2, cap - 1, 65, cap // 3)[i % 8] for i in range(b)]


CASES = [  # b, cap, heads, kv_heads, window, sinks
    (2, 600, 8, 2, 300, 4),      # few outputs, slices
    (24, 600, 32, 8, 300, 4),    # many outputs, slices
    (40, 600, 8, 8, 600, 0),     # 320 items of up to 600 keys, not cut
    (17, 900, 16, 2, 500, 1),    # groups of 8: the rests fill all their rows
    (9, 700, 36, 4, 256, 3),     # groups of 9: a product of their own
    (40, 300, 80, 8, 300, 0),    # groups of 10, not cut
    (13, 500, 20, 1, 90, 100),   # groups of 20: 16 heads and 4
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%dc%dh%d_%dw%ds%d" % c)
def test_one_rounding_whatever_the_batch(case, d, dt):
    b, cap, heads, kv, window, sinks = case
    lens = lengths(b, cap)
    Q, K, V = make(b, cap, heads, kv, d, dt, lens, seed=b + d)
    O, LSE = call(Q, K, V, lens, heads, kv, window, sinks)
    ref, tO, lse, tl = reference(Q, K, V, lens, heads, kv, window, sinks)
    close(O, ref, tO, "O")
    close(LSE, lse, tl, "LSE")


def test_a_sequence_does_not_depend_on_its_batch():
    """The same request in batches of 320 and of 400 items, neither cut into
    slices: bit for bit the same answer; and within the bound alone."""
    heads, kv, d, cap, window = 8, 8, 128, 700, 700
    lens = lengths(50, cap)
    Q, K, V = make(50, cap, heads, kv, d, BF, lens, 3)
    big, lse = call(Q, K, V, lens, heads, kv, window, 0)
    part, lse2 = call(Q[:40], K[:40], V[:40], lens[:40], heads, kv, window, 0)
    assert torch.equal(big[:40], part) and torch.equal(lse[:40], lse2)
    ref, tO, _, _ = reference(Q, K, V, lens, heads, kv, window, 0)
    for i in (2, 4, 5):
        one, _ = call(Q[i:i + 1], K[i:i + 1], V[i:i + 1], lens[i:i + 1], heads, kv, window, 0)
        close(one, ref[i:i + 1], tO[i:i + 1], f"alone {i}")
