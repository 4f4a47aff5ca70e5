"""What the attention of drafted tokens plans, on the CPU: its workspace, and the
form that calls take (a change of that choice has to show here, or it would move
the GPU tests from one kernel to the other unseen)."""

import pytest

import weight_activation_quantized_amd as mq

workspace, form = mq.kv8_tree_attention_workspace_bytes, mq.kv8_tree_attention_form


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


def test_nothing_to_do_and_refusals():
    assert form(0, 1, 8, 2, 128, 64, 10, 1) is None and form(4, 0, 8, 2, 128, 64, 10, 1) is None
    assert form(4, 4, 7, 2, 128, 64, 10, 1) is None and form(4, 4, 8, 2, 96, 64, 10, 1) is None
    assert form(4, 4, 8, 2, 128, 64, 0, 1) is None and form(2000, 1, 8, 2, 128, 64, 100, 1025) is None
    assert form(2000, 2, 8, 2, 128, 64, 100, 1024) is not None


@pytest.mark.parametrize("width", [1, 100, 16384])
@pytest.mark.parametrize("batch", [1, 64, 4096])
def test_few_rows_a_head(batch, width):
    assert form(batch * 16, batch, 32, 8, 128, 64, width, 16) == "decode"
    assert form(batch * 8, batch, 56, 7, 64, 16, width, 8) == "decode"


def test_calls_of_the_gpu_tests():
    """Trees of test_gpu_tree.py in wide tables, and those that its names do not tell."""
    for page in (16, 128):
        assert form(93, 2, 6, 2, 128, page, 65536 // page, 90) == "prompt"
    assert form(120, 2, 8, 2, 128, 16, 4096, 90) == "prompt" and form(170, 5, 8, 2, 128, 16, 4096, 100) == "prompt"
    assert form(130, 2, 4, 2, 128, 16, 4096, 90) == "prompt" and form(170, 2, 8, 2, 64, 16, 4096, 150) == "prompt"
    assert form(84, 2, 4, 1, 128, 64, 142, 64) == "decode"  # the long contexts of that file
    assert form(200, 1, 4, 1, 64, 32, 189, 200) == "decode"
    assert form(2300, 150, 4, 1, 64, 64, 512, 300) == "prompt"
    assert form(36, 3, 8, 2, 64, 16, 10, 30) == "decode"  # the drafted steps
