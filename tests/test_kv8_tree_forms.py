"""What the attention of drafted tokens plans, on the CPU: its workspace."""

import pytest

import weight_activation_quantized_amd as mq

workspace = mq.kv8_tree_attention_workspace_bytes


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs,new,Hq,Hkv,tokens", [(64, 64, 32, 8, 4096), (256, 17, 32, 8, 4096), (1024, 17, 32, 8, 2048),
                                                    (4096, 17, 32, 8, 1024), (65535, 17, 32, 8, 512), (65535, 17, 8, 8, 512),
                                                    (300, 1024, 64, 1, 2048), (200, 33, 96, 12, 100000), (40, 9, 1024, 128, 64000)])
def test_workspace_is_bounded(seqs, new, Hq, Hkv, tokens, D):
    """Parts of at most 1024 shares of 256 rows, with their maxima and sums, and 8
    bytes a row, whatever the batch."""
    T = seqs * new
    need = workspace(T, seqs, Hq, Hkv, D, 64, -(-tokens // 64), new)
    assert need <= 1024 * 256 * (D + 2) * 4 + 8 * T * Hq
