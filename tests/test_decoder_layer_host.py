"""Workspace queries of the decoder-layer operators for calls that do nothing
(no GPU)."""
import pytest

from megatron_tensor_transformer_logical_b200 import binding as L


def test_no_tokens_need_a_workspace_like_any_other():
    """tp_qk_norm_rope_bwd takes M = 0, so its workspace can be asked for."""
    size = lambda M, d=64, dt=L.TP_BF16: L.load().tp_workspace_size(L.TP_OP_QK_NORM_ROPE_BWD, M, d,
                                                                     0, 0, 1, dt)
    assert size(0) == size(1) == size(1 << 20) > 0  # depends on d only
    assert size(0, dt=L.TP_F16) == size(0)
    assert size(-1) == 0 and size(0, 0) == 0 and size(0, 264) == 0
    assert L.qk_norm_rope_workspace(0, 64, "cpu").numel() == size(0)
    with pytest.raises(L.TPError):
        L.qk_norm_rope_workspace(-1, 64, "cpu")
