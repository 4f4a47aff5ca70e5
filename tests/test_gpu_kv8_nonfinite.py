"""NaN and infinities in the paged e4m3 cache's inputs: what is not a number is
never turned into one, whatever form and number of splits a call takes, and does
not reach other sequences."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import half_tensor
from tests.kv8_util import append, attend, empty_cache

pytestmark = pytest.mark.gpu

# new tokens of each of two sequences, their keys, table width in pages of 64:
# unsplit decode of four and eight wavefronts, split decode, prompts split and not
FORMS = {"decode": (1, 200, 4, 2), "decode, eight wavefronts": (1, 500, 8, 2), "decode, split": (1, 5000, 100, 2),
         "decode of five, split": (5, 2000, 64, 2), "prompt, split": (90, 3000, 2048, 2), "prompt": (64, 700, 512, 128)}


def _two(rng, form, D, half):
    """Two sequences (the second one plain) of a form and their dense inputs."""
    new, keys, width, Hkv = FORMS[form]
    n = -(-keys // 64)
    cache = empty_cache(2 * n, Hkv, 64, D)
    cache[0][:] = o8.e4m3_encode(np.clip(rng.standard_normal(cache[0].shape) * 60, -448, 448))
    cache[1][:] = o8.e4m3_encode(np.clip(rng.standard_normal(cache[1].shape) * 60, -448, 448))
    table = np.full((2, width), -1, np.int32)
    table[:, :n] = rng.permutation(2 * n).reshape(2, n)
    tq, _ = half_tensor(rng.standard_normal((2 * new, 4 * Hkv, D)), half)
    needs = mq.kv8_attention_workspace_bytes(2 * new, 2, 4 * Hkv, Hkv, D, 64, width, new)
    assert (needs > 0) == ("split" in form)
    return new, keys, cache, table, tq


@pytest.mark.parametrize("half,D", [("fp16", 64), ("bf16", 128)])
@pytest.mark.parametrize("form", FORMS)
def test_nan_in_a_row_of_q(form, D, half):
    rng = np.random.default_rng(1)
    new, keys, cache, table, tq = _two(rng, form, D, half)
    args = cache, table, [0, new, 2 * new], [keys, keys]
    plain = attend(tq, *args, f"{form}: finite")
    assert np.isfinite(plain).all()
    tq[new - 1, 1, 3] = float("nan")
    got = attend(tq, *args, f"{form}: NaN in q")
    bad = np.isnan(got)
    assert bad[new - 1, 1].all()
    bad[new - 1, 1] = False
    assert not bad.any() and np.array_equal(got[~np.isnan(got)], plain[~np.isnan(got)])


@pytest.mark.parametrize("half,D", [("fp16", 64), ("bf16", 128)])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("at", [0, 100, -1])
def test_nan_codes(form, at, D, half):
    """One K code: every row that sees its token, all dimensions; one V code: that
    dimension of them. The other head and the other sequence keep every bit."""
    rng = np.random.default_rng(2)
    new, keys, cache, table, tq = _two(rng, form, D, half)
    cu, lens = [0, new, 2 * new], [keys, keys]
    plain = attend(tq, cache, table, cu, lens, f"{form}: finite")
    t = keys - 1 if at < 0 else at
    first = max(t - (keys - new), 0)  # rows from here on see it
    p = table[0, t // 64]
    for what in ("K", "V"):
        c = [a.copy() for a in cache]
        if what == "K":
            c[0][p, 1, t % 64, 5] = 0x7F
        else:
            c[1][p, 1, 5, t % 64] = 0xFF
        got = attend(tq, c, table, cu, lens, f"{form}: NaN {what} code of token {t}")
        bad = np.isnan(got)
        assert bad[first:new, 4:8][..., slice(None) if what == "K" else 5].all()
        assert np.array_equal(got[new:], plain[new:])
        others = np.delete(np.arange(tq.shape[1]), np.arange(4, 8))
        assert np.array_equal(got[:new, others], plain[:new, others])
        if what == "V":
            assert np.array_equal(np.delete(got, 5, 2), np.delete(plain, 5, 2))


@pytest.mark.parametrize("half,D", [("fp16", 64), ("bf16", 128)])
@pytest.mark.parametrize("form", FORMS)
def test_nan_scales(form, D, half):
    """A page's scale of K or V: every row that sees one of its tokens."""
    rng = np.random.default_rng(3)
    new, keys, cache, table, tq = _two(rng, form, D, half)
    cu, lens = [0, new, 2 * new], [keys, keys]
    plain = attend(tq, cache, table, cu, lens, f"{form}: finite")
    for which in (2, 3):
        c = [a.copy() for a in cache]
        c[which][table[0, 1], 1] = np.nan
        got = attend(tq, c, table, cu, lens, f"{form}: NaN scale {which}")
        assert np.isnan(got[:new, 4:8]).all()
        assert np.array_equal(got[new:], plain[new:])
        others = np.delete(np.arange(tq.shape[1]), np.arange(4, 8))
        assert np.array_equal(got[:new, others], plain[:new, others])


@pytest.mark.parametrize("half,D", [("fp16", 64), ("bf16", 128)])
@pytest.mark.parametrize("form", FORMS)
def test_what_no_row_sees_may_be_nan(form, D, half):
    """Page 0, which unknown page numbers and tiles past the end read in their
    place, and everything behind the last tokens: NaN codes and scales there
    change no bit."""
    rng = np.random.default_rng(4)
    new, keys, cache, table, tq = _two(rng, form, D, half)
    P, H = cache[2].shape
    table = np.where(table >= 0, table + 1, table)
    table[1, 0] = P + 1  # of no pool: the second sequence misses its first page
    c = [np.concatenate([a[:1], a]) for a in cache]
    args = table, [0, new, 2 * new], [keys, keys - 7]
    plain = attend(tq, c, *args, f"{form}: finite")
    c[0][0], c[1][0], c[2][0], c[3][0] = 0x7F, 0x7F, np.nan, np.nan
    for b, n in enumerate(args[2]):
        if n % 64:
            p = table[b, n // 64]
            c[0][p, :, n % 64:] = 0xFF
            c[1][p, :, :, n % 64:] = 0xFF
    got = attend(tq, c, *args, f"{form}: NaN that no row sees")
    assert np.isfinite(plain).all() and np.array_equal(got, plain)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("news,olds", [([1, 1, 1], [0, 5, 15]), ([3, 2, 40], [0, 13, 3]), ([130, 64, 200], [0, 9, 130])])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_append_of_what_is_not_finite(D, page, news, olds, half):
    """NaN and both infinities among the new tokens, NaN codes among the older
    ones whose page changes its scale: bit for bit, each spoils itself only."""
    rng = np.random.default_rng(page + D + sum(news))
    totals = [n + o for n, o in zip(news, olds)]
    T, H = sum(news), 2
    P = sum(-(-t // page) for t in totals)
    table = np.full((3, 40), -1, np.int32)
    at = 0
    for b, t in enumerate(totals):
        n = -(-t // page)
        table[b, :n] = range(at, at + n)
        at += n
    cache = empty_cache(P, H, page, D, 2.0 ** -9)
    for c in cache[:2]:
        c[:] = o8.e4m3_encode(np.clip(rng.standard_normal(c.shape) * 90, -448, 448))
        c.reshape(-1)[::37] = 0x7F
        c.reshape(-1)[5::41] = 0xFF
    k, v = (rng.standard_normal((T, H, D)) * 3 for _ in range(2))
    for x in (k, v):
        for bad in (np.nan, np.inf, -np.inf):
            x[rng.integers(0, T, 3), rng.integers(0, H, 3), rng.integers(0, D, 3)] = bad
        x[0, 0, :] = np.inf  # a token of nothing else
    append(k, v, half, cache, table, news, totals, "not finite")
