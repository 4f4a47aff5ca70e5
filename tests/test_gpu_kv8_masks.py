"""Which keys a row of attention sees, to the key: against the rows' own bounds
(``oracle.fp8.kv8_attention_rows``; CPU tests show that they reject a lost or an
extra key on these inputs), and by counting. Both forms, split and not."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from tests.fp8_util import half_tensor
from tests.kv8_util import attend, check_rows, counted, paged, planted

pytestmark = pytest.mark.gpu

FRO = {"fp16": 1e-3, "bf16": 5e-3}
LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 1300]
# new tokens, all tokens, kv heads, heads of a group, tokens that a table can hold (0: as needed), form, split
CALLS = {
    "single tokens": ([1] * 16, LENS, 2, 4, 0, "decode", True),
    "single tokens, short": ([1] * 12, LENS[:12], 2, 4, 0, "decode", False),
    "single tokens, eight wavefronts": ([1, 1], [500, 257], 2, 8, 0, "decode", False),
    "single tokens, many splits": ([1, 1], [5000, 70], 1, 4, 0, "decode", True),
    "a few": ([2, 0, 5, 16, 3], [2, 9, 67, 528, 1029], 2, 4, 0, "decode", True),
    "small prompt": ([100, 1, 64, 65], [100, 50, 200, 65], 2, 4, 0, "decode", False),
    "prompt, split": ([100, 1, 64, 65, 0], [100, 50, 200, 65, 7], 2, 4, 65536, "prompt", True),
    "prompt, more new than cached": ([70, 90], [40, 0], 2, 4, 65536, "prompt", True),
    "prompt, groups of three": ([130], [700], 2, 3, 65536, "prompt", True),
    "prompt": ([64, 1, 50], [700, 64, 190], 86, 4, 704, "prompt", False),
}


def _call(name, page, D):
    news, totals, Hkv, G, wide, form, split = CALLS[name]
    width = -(-wide // page) if wide else -(-(max(totals) + 1) // page)
    sizes = sum(news), len(news), Hkv * G, Hkv, D, page, width, max(news)
    assert mq.kv8_attention_form(*sizes) == form
    assert (mq.kv8_attention_workspace_bytes(*sizes) > 0) == split
    return news, totals, Hkv, G, width, np.concatenate([[0], np.cumsum(news)])


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("name", [n for n in CALLS if n != "prompt"])
def test_rows(name, page, D, half):
    rng = np.random.default_rng(page + D)
    news, totals, Hkv, G, width, cu = _call(name, page, D)
    cache, table = paged(rng, totals, Hkv, page, D, width)
    check_rows(rng.standard_normal((sum(news), Hkv * G, D)), half, cache, table, cu, totals, name, fro=FRO[half])


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("prompt", "prompt, more new than cached")])
def test_peaked_rows(name, page, D, half):
    """The last key has nearly all of the weight, the one behind it would have more."""
    rng = np.random.default_rng(page + D + 1)
    news, totals, Hkv, G, width, cu = _call(name, page, D)
    q, cache, table = planted(rng, news, totals, Hkv, G, D, page, width)
    check_rows(q, half, cache, table, cu, totals, name)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D,page", [(64, 64), (128, 16), (128, 128)])
@pytest.mark.parametrize("name", CALLS)
def test_counted_keys(name, page, D, half):
    """Equal weights and one-hot values: the output is a count over a count, in
    binary32 but for a reciprocal and a product (2^-23 each), rounded once."""
    rng = np.random.default_rng(page + D + 2)
    news, totals, Hkv, G, width, cu = _call(name, page, D)
    q, cache, table, want = counted(rng, news, totals, Hkv, G, D, page, width)
    got = attend(half_tensor(q, half)[0], cache, table, cu, totals, name, scale=0.0)
    u = 2.0 ** -8 if half == "bf16" else 2.0 ** -11
    assert np.all(np.abs(got - want) <= (u + 2.0 ** -20) * want)
