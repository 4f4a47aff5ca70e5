"""Attention where nearly all of the softmax lies on one key with a small value
(the first key of a long context is often such): the many small weights beside
it make up the output and must not be lost to the 16-bit product."""

import numpy as np
import pytest

from oracle import fp8 as o8
from tests.kv8_util import check_rows, empty_cache

pytestmark = pytest.mark.gpu


def _sink(rng, keys, news, Hkv, G, D, page, gap, sink_at, width=None, vscale=(4, 4)):
    """Every key has the score 0 but one, `gap` (base 2) above; that one has the
    value 0 (in a page of scale 2^vscale[1]), the others values around 1."""
    n = -(-keys // page)
    cache = empty_cache(n + 2, Hkv, page, D)
    table = np.full((1, width or n), -1, np.int32)
    table[0, :n] = rng.permutation(n + 2)[:n]
    cache[1][:] = o8.e4m3_encode(64 * rng.uniform(0.5, 1.5, cache[1].shape))
    cache[3][:] = 2.0 ** vscale[0]
    p, t = table[0, sink_at // page], sink_at % page
    cache[3][p] = 2.0 ** vscale[1]
    cache[1][p, :, :, t] = 0
    # q is 1 everywhere and softmax_scale 1: score = D * code * 2^-6
    q = np.ones((news, Hkv * G, D))
    want = gap * np.log(2) / D / 2.0 ** -6
    cache[0][p, :, t] = o8.e4m3_encode(want)
    return q, cache, table


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("keys,gap", [(1000, 26), (5000, 26), (32768, 24), (131072, 26)])
@pytest.mark.parametrize("sink_at", [0, 900])
def test_single_tokens(keys, gap, sink_at, half):
    rng = np.random.default_rng(keys + gap)
    q, cache, table = _sink(rng, keys, 1, 1, 4, 128, 64, gap, sink_at)
    check_rows(q, half, cache, table, [0, 1], [keys], f"sink at {sink_at}", scale=1.0)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keys,gap,sink_at", [(3000, 26, 0), (9000, 24, 0), (9000, 26, 4000)])
def test_prompts(keys, gap, sink_at, D, half):
    """200 rows per kv head under tables wide enough for the prompt form."""
    rng = np.random.default_rng(keys + gap)
    q, cache, table = _sink(rng, keys, 50, 1, 4, D, 64, gap, sink_at, width=8192)
    check_rows(q, half, cache, table, [0, 50], [keys], f"sink at {sink_at}, prompt", scale=1.0)


@pytest.mark.parametrize("news,width", [(1, None), (50, 8192)])
def test_sink_in_a_page_of_larger_values(news, width):
    """The sink's page has a V scale 2^8 times the others': its weight counts for
    as much more in the reference of the exponents."""
    rng = np.random.default_rng(5)
    q, cache, table = _sink(rng, 9000, news, 2, 4, 128, 16, 18, 0, width=width, vscale=(4, 12))
    check_rows(q, "bf16", cache, table, [0, news], [9000], "larger page", scale=1.0)


@pytest.mark.parametrize("news,width", [(1, None), (50, 8192)])
def test_values_of_zero(news, width):
    """Pages of the smallest scale, as zeros leave them, under many keys: the sum
    of the weights stays within binary32 and the output is 0."""
    rng = np.random.default_rng(6)
    q, cache, table = _sink(rng, 20000, news, 1, 4, 128, 64, 0, 0, width=width, vscale=(-100, -100))
    cache[1][:] = 0
    got = check_rows(q, "bf16", cache, table, [0, news], [20000], "zeros", scale=1.0)
    assert not got.any()
    cache[1][:] = 0x38  # 1.0: 2^-100 in bf16
    got = check_rows(q, "bf16", cache, table, [0, news], [20000], "tiny", scale=1.0)
    assert np.all(got == 2.0 ** -100)


@pytest.mark.parametrize("exponent", [114, 117, 120])
@pytest.mark.parametrize("news,width", [(1, None), (50, 8192)])
def test_largest_scales(news, width, exponent):
    """V scales at the upper end of their range: sums of weights over them are
    small, and neither they nor their reciprocals are lost."""
    rng = np.random.default_rng(8)
    q, cache, table = _sink(rng, 3000, news, 1, 4, 128, 64, 3, 0, width=width, vscale=(exponent, exponent))
    cache[1][:] = o8.e4m3_encode(rng.uniform(0.5, 100, cache[1].shape))
    check_rows(q, "bf16", cache, table, [0, news], [3000], "largest scales", scale=1.0)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("news,width", [(1, None), (50, 8192)])
def test_zero_values_beside_large_ones(news, width, half):
    """Every other page holds zeros alone (scale 2^-100, as the append leaves
    them), the others values of scale 2^0; the scores are the same everywhere, so
    half of the sum of the weights comes from weights 2^-100 of the largest."""
    rng = np.random.default_rng(7)
    q, cache, table = _sink(rng, 9000, news, 1, 4, 128, 64, 0, 0, width=width, vscale=(0, 0))
    for p in table[0, :141:2]:
        cache[1][p], cache[3][p] = 0, 2.0 ** -100
    check_rows(q, half, cache, table, [0, news], [9000], "zeros beside", scale=1.0)
