"""NaN tokens in window attention (GPU): a NaN score shows in the O and the LSE of
every query that sees it and in no other's, it never becomes the zero of a query
that sees nothing."""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu
from tests.test_gpu_window import BF, FP, make, run, visible

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


@pytest.mark.parametrize("sq,sk,window,sinks", [(400, 400, 60, 4), (400, 400, 400, 0),
                                                (300, 700, 90, 130), (500, 200, 40, 2)])
@pytest.mark.parametrize("d,dt", [(64, FP), (128, BF)])
def test_nan_queries_and_keys(sq, sk, window, sinks, d, dt):
    b, heads, kv = 2, 4, 2
    Q, K, V, _ = make(b, sq, sk, heads, kv, d, dt, 31)
    clean = run(Q, K, V, None, b, heads, kv, window, sinks)
    seen = visible(sq, sk, window, sinks)

    def check(got, nan):  # nan [b, heads, sq]
        per_row = nan.transpose(1, 2).reshape(b * sq, heads, 1).expand(-1, -1, d).reshape(
            b * sq, heads * d)
        assert torch.equal(torch.isnan(got["O"]), per_row)
        assert torch.equal(got["O"][~per_row], clean["O"][~per_row])
        assert torch.equal(torch.isnan(got["LSE"]), nan)
        assert torch.equal(got["LSE"][~nan], clean["LSE"][~nan])

    bad, nan = Q.clone(), torch.zeros(b, heads, sq, dtype=torch.bool, device="cuda")
    for i, h, r in ((0, 1, sq - 1), (0, 2, sq // 2), (1, 0, 0), (1, 3, sq - 130)):
        bad[i * sq + r, h * d + 5] = NAN
        nan[i, h, r] = seen[r].any()
    check(run(bad, K, V, None, b, heads, kv, window, sinks), nan)
    bad, nan = K.clone(), torch.zeros_like(nan)
    for i, g, c in ((0, 1, sk // 2), (1, 0, 1), (1, 1, sk - 1)):
        bad[i * sk + c, g * d + 7] = NAN
        nan[i, g * 2:g * 2 + 2] |= seen[:, c]
    check(run(Q, bad, V, None, b, heads, kv, window, sinks), nan)


@pytest.mark.parametrize("b,heads,kv", [(3, 8, 2), (3, 36, 4), (41, 8, 8)])
@pytest.mark.parametrize("d,dt", [(64, BF), (128, FP)])
def test_nan_in_a_decoding_step(b, heads, kv, d, dt):
    """Cut into slices and not, few and many query heads on a key head."""
    cap, window, sinks, G = 900, 700, 3, heads // kv
    g = torch.Generator(device="cuda").manual_seed(32)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    Q, K, V = rn(b, heads * d), rn(b, cap, kv * d), rn(b, cap, kv * d)
    lens = torch.full((b,), 850, dtype=torch.int32, device="cuda")
    lens[1] = 0
    ws = L.window_attn_decode_workspace(b, cap, heads, kv, d, window, sinks)

    def call(Q, K):
        O, LSE = torch.empty_like(Q), torch.empty(b, heads, device="cuda")
        L.tp_window_attn_decode(Q, K, V, lens, O, LSE, heads, kv, window, sinks, ws)
        return O.reshape(b, heads, d), LSE

    O, LSE = call(Q, K)
    assert not torch.isnan(O).any() and (O[1] == 0).all() and (LSE[1] == float("-inf")).all()
    badq, badk = Q.clone(), K.clone()
    badq[2, (heads - 1) * d] = NAN
    badq[1] = NAN                      # sees nothing
    badk[0, 500, 0] = NAN
    badk[2, 100, 0] = NAN              # hidden: before the window
    badk[2, 860, 0] = NAN              # past the end
    nan = torch.zeros(b, heads, dtype=torch.bool, device="cuda")
    nan[2, heads - 1], nan[0, :G] = True, True
    O2, LSE2 = call(badq, badk)
    assert torch.equal(torch.isnan(LSE2), nan) and torch.equal(LSE2[~nan], LSE[~nan])
    assert torch.isnan(O2[nan]).all() and torch.equal(O2[~nan], O[~nan])
