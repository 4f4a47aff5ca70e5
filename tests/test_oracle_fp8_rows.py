"""Pins of the e4m3 cache's oracle: what is not finite in an append; the rows'
error bound of attention, which must not let through an output that lost each
row's last key or saw one more."""

import numpy as np
import pytest

from oracle import fp8 as o
from tests import kv8_util as u


def test_append_of_what_is_not_finite():
    # one page of 4 tokens, one head, three dimensions; the older token holds NaN
    kc, vc = np.zeros((1, 1, 4, 3), np.uint8), np.zeros((1, 1, 3, 4), np.uint8)
    kc[0, 0, 0] = vc[0, 0, :, 0] = [0xFF, 0x38, 0x7F]  # NaN, 1, NaN
    ks, vs = np.ones((1, 1), np.float32), np.ones((1, 1), np.float32)
    x = np.float32([[[np.inf, 896.0, np.nan]], [[-np.inf, 2.0, 4.0]]])
    a = o.kv8_append_ref(x, x, kc, vc, ks, vs, np.zeros((1, 1), np.int32), [0, 2], [3])
    assert a[2][0, 0] == 2.0 and a[3][0, 0] == 2.0  # 896 decides, not the infinity
    for codes in (a[0][0, 0], a[1][0, 0].T):
        assert codes[0].tolist() == [0xFF, 0x30, 0x7F]  # 0.5: moved to the new scale; NaN as it was
        assert codes[1].tolist() == [0x7F, 0x7E, 0x7F]
        assert codes[2].tolist() == [0x7F, 0x38, 0x40]
        assert not codes[3].any()
    y = np.float32([[[np.nan, np.inf, -np.inf]]])
    b = o.kv8_append_ref(y, y, kc, vc, ks, vs, np.zeros((1, 1), np.int32), [0, 1], [1])
    assert b[2][0, 0] == np.float32(2.0 ** -100) and b[0][0, 0, 0].tolist() == [0x7F] * 3


FRO = {"fp16": 1e-3, "bf16": 5e-3}


def _rejected(q, half, cache, table, cu, lens, by, fro):
    """Sequences whose rows, each seeing `by` keys more, pass the check: none may."""
    q = o.round_half(q, half)
    scale = q.shape[2] ** -0.5
    o64, bound = o.kv8_attention_rows(q, *cache, table, cu, lens, scale, half)
    with np.errstate(invalid="ignore"):  # (a NaN code behind the last token)
        off, _, _ = o.kv8_attention_ref(q, *cache, table, cu, np.maximum(np.array(lens) + by, 0), scale)
    passes = []
    for b in range(len(lens)):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        within = np.all(np.abs(off[rows] - o64[rows]) <= bound[rows])
        size = np.linalg.norm(o64[rows])
        if within and not (fro and np.linalg.norm(off[rows] - o64[rows]) > fro * size):
            passes.append(lens[b])
    return passes


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("by", [-1, 1])
def test_bound_pins_the_mask(by, D, half):
    rng = np.random.default_rng(D + by)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 1300]
    cache, table = u.paged(rng, lens, 2, 16, D)
    q = rng.standard_normal((len(lens), 8, D))
    assert _rejected(q, half, cache, table, np.arange(len(lens) + 1), lens, by, FRO[half]) == []


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("by", [-1, 1])
def test_bound_pins_the_mask_of_peaked_rows(by, D, half):
    """By the elements' bound alone."""
    rng = np.random.default_rng(D + by)
    news, lens = [1, 1, 3, 20, 1], [333, 900, 500, 64, 5000]
    q, cache, table = u.planted(rng, news, lens, 2, 4, D, 64)
    assert _rejected(q, half, cache, table, np.concatenate([[0], np.cumsum(news)]), lens, by, None) == []


def test_bound_holds_the_kernel_s_roundings():
    """The second product with weights rounded to fp16 as the kernels round them,
    the first in binary32: within the bound, and not by so much that it says
    nothing."""
    rng = np.random.default_rng(5)
    L, D = 700, 128
    cache, table = u.paged(rng, [L], 2, 16, D)
    q = o.round_half(rng.standard_normal((1, 8, D)), "fp16")
    o64, bound = o.kv8_attention_rows(q, *cache, table, [0, 1], [L], D ** -0.5, "fp16")
    pos = np.arange(L)
    ids = table[0, pos // 16]
    worst = 0
    for hq in range(8):
        h = hq // 4
        k = (o.e4m3_decode(cache[0][ids, h, pos % 16]) * cache[2][ids, h][:, None]).astype(np.float32)
        v, vs = o.e4m3_decode(cache[1][ids, h, :, pos % 16]), cache[3][ids, h].astype(np.float64)
        x = (k @ q[0, hq]) * np.float32(D ** -0.5 * np.log2(np.e)) + np.log2(vs).astype(np.float32)
        w = np.exp2(x - x.max() + np.float32(15))
        got = (w.astype(np.float16).astype(np.float64) @ v) / (w.astype(np.float64) / vs).sum()
        err = np.abs(got.astype(np.float16).astype(np.float64) - o64[0, hq]) / bound[0, hq]
        assert np.all(err <= 1)
        worst = max(worst, err.max())
    assert worst > 0.05
