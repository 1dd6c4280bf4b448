"""The work that the profile reports for window attention (GPU): 4 d flops per
visible (query, key) pair forward, 10 d backward, counted here one by one."""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu
from tests.test_gpu_window import BF, make, run, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


@pytest.mark.parametrize("b,sq,sk,heads,kv,d,window,sinks", [
    (1, 385, 385, 4, 4, 64, 64, 300),    # many sinks: rows between window and both
    (2, 200, 200, 2, 1, 128, 50, 200),   # sinks up to the end: full causal
    (1, 300, 300, 2, 2, 64, 300, 0),
    (1, 300, 300, 2, 2, 64, 1, 0),
    (2, 70, 700, 4, 1, 64, 90, 1),       # queries at the end
    (1, 5, 700, 2, 1, 64, 200, 600),
    (2, 300, 170, 2, 1, 128, 40, 20),    # first queries see nothing
    (1, 600, 130, 2, 2, 64, 500, 4),
])
def test_visible_pairs(b, sq, sk, heads, kv, d, window, sinks):
    Q, K, V, dO = make(b, sq, sk, heads, kv, d, BF)
    L.tp_profile_enable(True)
    try:
        run(Q, K, V, dO, b, heads, kv, window, sinks)
        torch.cuda.synchronize()
        fwd, bwd = (L.tp_profile_read(k)["flops"] for k in (L.TP_KIND_ATTN_FWD,
                                                            L.TP_KIND_ATTN_BWD))
    finally:
        L.tp_profile_enable(False)
    pairs = visible(sq, sk, window, sinks).sum().item() * b * heads
    assert (fwd, bwd) == (4.0 * d * pairs, 10.0 * d * pairs)
