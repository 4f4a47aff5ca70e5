"""Which form of attention the GPU tests' calls take, on the CPU: a change of
that choice has to show here, or it would move tests from one kernel to the
other unseen."""

import pytest

import weight_activation_quantized_amd as mq

form, workspace = mq.kv8_attention_form, mq.kv8_attention_workspace_bytes


def test_nothing_to_do_and_refusals():
    assert form(0, 1, 8, 2, 128, 64, 10, 1) is None and form(4, 0, 8, 2, 128, 64, 10, 1) is None
    assert form(4, 4, 7, 2, 128, 64, 10, 1) is None and form(4, 4, 8, 2, 96, 64, 10, 1) is None
    assert form(4, 4, 8, 2, 128, 48, 10, 1) is None and form(4, 4, 8, 2, 128, 64, 0, 1) is None


@pytest.mark.parametrize("width", [1, 100, 16384])
@pytest.mark.parametrize("batch", [1, 64, 4096])
def test_single_tokens(batch, width):
    assert form(batch, batch, 32, 8, 128, 64, width, 1) == "decode"
    assert form(batch, batch, 64, 1, 64, 16, width, 1) == "decode"


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_in_wide_tables(D, page):
    """The calls of the GPU test of that name."""
    assert form(230, 4, 8, 2, D, page, 65536 // page, 100) == "prompt"
    assert form(122, 3, 6, 2, D, page, 65536 // page, 90) == "prompt"
    assert form(300, 1, 5, 1, D, page, 65536 // page, 300) == "prompt"


def test_large_prompts():
    assert form(2029, 2, 32, 4, 128, 64, 24, 1030) == "prompt"
    assert form(1490, 3, 16, 4, 128, 64, 32, 777) == "prompt"
    for page in (16, 128):
        assert form(366, 2, 256, 8, 64, page, -(-3400 // page), 300) == "prompt"
    assert form(93, 2, 4, 2, 128, 16, 4096, 90) == "prompt"
    assert form(250, 1, 8, 2, 128, 16, 4096, 250) == "prompt" and form(270, 2, 8, 2, 128, 16, 4096, 200) == "prompt"
    assert form(200, 1, 4, 1, 64, 64, 8192, 50) == "prompt"  # the tests of small weights


def test_small_prompts_go_with_single_tokens():
    """A prompt workgroup walks its keys one tile after the other: calls of few
    row tiles times keys are left to the other form."""
    assert form(100, 1, 32, 8, 128, 64, 3, 100) == "decode"
    assert form(120, 3, 8, 2, 128, 16, 100, 40) == "decode"
    assert form(300, 1, 4, 1, 128, 64, 141, 300) == "decode"
