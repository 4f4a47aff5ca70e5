"""Keeping a path of drafted tokens in the e4m3 cache on an MI355X: every byte and
scale of every layer against the oracle, moves within a page and across pages
of other scales, paths that end early, pages that must stay as they are."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import drafts as od
from tests.draft_util import layered, offsets, up
from tests.fp8_util import codes_of, codes_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu


def check(rng, news, totals, paths, H, D, page, what, layers=2, cache=None, table=None, kept=None, width=None):
    if cache is None:
        cache, table = layered(rng, layers, [max(t, 1) for t in totals], H, page, D)
    layers = cache[0].shape[0]
    width = width or max(max(news), 1)
    path = np.full((len(news), width), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    kept = np.array([len(p) for p in paths] if kept is None else kept, np.int32)
    cu, lens = offsets(news), np.array(totals, np.int32)
    announce(f"kv8_tree_keep {what} {cache[0].shape} new={list(news)[:4]} total={totals[:4]} kept={kept[:4].tolist()}")
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    if layers == 1:
        mq.kv8_tree_keep(*[t[0] for t in dev], up(table), up(cu), up(lens), up(path), up(kept))
    else:
        mq.kv8_tree_keep(*dev, up(table), up(cu), up(lens), up(path), up(kept))
    want = od.keep_ref(*cache, table, cu, lens, path, kept)
    for name, a, b in zip(("K codes", "V codes", "K scales", "V scales"), dev, want):
        got = codes_of(a) if b.dtype == np.uint8 else host(a).view(np.uint32)
        bad = np.argwhere(got != (b if b.dtype == np.uint8 else b.view(np.uint32)))
        assert bad.size == 0, f"{what}: {len(bad)} {name} differ, first at {bad[:3].tolist()}"
    return want


def ascending(rng, n, m):
    return [0] + sorted(1 + rng.choice(n - 1, m - 1, replace=False)) if m > 1 else [0]


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_paths(page, D, layers):
    rng = np.random.default_rng(page + D)
    news = [8, 64, 26, 1, 200]
    totals = [n + t for n, t in zip(news, (0, page - 3, 77, 5, 300))]
    paths = [ascending(rng, n, m) for n, m in zip(news, (3, 9, 26, 1, 120))]
    check(rng, news, totals, paths, 2, D, page, "paths", layers)


def test_nothing_moves():
    rng = np.random.default_rng(1)
    news, totals = [5, 8, 0], [20, 33, 9]
    for paths, kept in (([[0], [0], []], None), ([list(range(5)), list(range(8)), []], None), ([[], [], []], [0, -3, 4])):
        cache, table = layered(rng, 2, totals, 2, 16, 64)
        want = check(rng, news, totals, paths, 2, 64, 16, "nothing moves", cache=cache, table=table, kept=kept)
        assert all(np.array_equal(a, b) for a, b in zip(want, cache))


def test_bad_paths_end():
    """Entries before their place or behind the new tokens end the path; counts
    beyond the new tokens and the path's width are cut."""
    rng = np.random.default_rng(2)
    news, totals = [8, 8, 8, 8], [30, 30, 8, 50]
    paths = [[0, 3, 1, 7], [0, 2, 8], [0, 4, -1, 6], [2 ** 31 - 1]]
    check(rng, news, totals, paths, 2, 64, 16, "bad paths")
    check(rng, news, totals, [[1, 2, 3, 4, 5, 6, 7]] * 4, 1, 64, 32, "cut", kept=[100, 8, 9, 7])
    check(rng, news, [4, 30, 0, 8], [[0, 2, 5]] * 4, 1, 64, 16, "more new tokens than cached")


def test_scales_far_apart_and_nan():
    """Sources whose scale is much larger (the page moves to it) or smaller (codes
    round away), NaN codes, which stay and count for no scale."""
    rng = np.random.default_rng(3)
    news, totals = [40, 40], [45, 52]
    for lo, hi in ((-30, 20), (-6, 3), (-100, 100)):
        cache, table = layered(rng, 2, totals, 2, 16, 64)
        for s in cache[2:]:
            s[:] = np.exp2(rng.integers(lo, hi, s.shape))
        for c in cache[:2]:
            c[rng.random(c.shape) < 0.02] = 0x7F
            c[rng.random(c.shape) < 0.02] = 0xFF
        check(rng, news, totals, [ascending(rng, 40, 12), ascending(rng, 40, 30)], 2, 64, 16, "far scales", cache=cache,
              table=table)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_sources_of_scales_that_are_not_finite(bad):
    """A token that its page's scale makes NaN or infinite is NaN where it moves to."""
    rng = np.random.default_rng(7)
    news, totals = [40, 40], [45, 52]
    cache, table = layered(rng, 2, totals, 2, 16, 64)
    for s in cache[2:]:
        s[:, table[0, 2], 0] = bad
        s[:, table[1, 3], 1] = bad
    paths = [[0, 5, 30, 33, 36], [0, 6, 7, 20, 38, 39]]
    want = check(rng, news, totals, paths, 2, 64, 16, f"scales of {bad}", cache=cache, table=table)
    assert (want[0][:, table[0, 0], 0, 7:10] == 0x7F).all()  # from nodes 30, 33 and 36, of page 2
    assert (want[1][:, table[1, 1], 1, :, :2] == 0x7F).all()  # from nodes 38 and 39, of page 3


def test_unknown_pages():
    rng = np.random.default_rng(4)
    news, totals = [30, 30], [40, 60]
    cache, table = layered(rng, 2, totals, 2, 16, 64)
    table[0, 1], table[1, 3] = -1, 2 ** 31 - 1
    paths = [ascending(rng, 30, 12), ascending(rng, 30, 14)]
    check(rng, news, totals, paths, 2, 64, 16, "unknown", cache=cache, table=table)
    check(rng, news, totals, paths, 2, 64, 16, "narrow table", cache=cache, table=table[:, :3].copy())


def test_many_sequences():
    rng = np.random.default_rng(5)
    news = [int(n) for n in rng.integers(0, 20, 90)]
    totals = [n + int(t) for n, t in zip(news, rng.integers(0, 40, 90))]
    check(rng, news, totals, [ascending(rng, n, int(rng.integers(1, n + 1))) if n else [] for n in news], 1, 64, 16, "many")


def test_refusals_of_the_wrapper():
    import torch
    rng = np.random.default_rng(6)
    cache, table = layered(rng, 2, [20], 2, 16, 64)
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    b = up(table), up(np.array([0, 4], np.int32)), up(np.array([20], np.int32))
    path, kept = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    mq.kv8_tree_keep(*dev, *b, path, kept)
    with pytest.raises(ValueError):
        mq.kv8_tree_keep(dev[0], dev[1][0], *dev[2:], *b, path, kept)
    with pytest.raises(ValueError):
        mq.kv8_tree_keep(dev[0], dev[1], dev[2][0], dev[3], *b, path, kept)
    with pytest.raises(ValueError):
        mq.kv8_tree_keep(*dev, *b, path, kept[:0])
    with pytest.raises(TypeError):
        mq.kv8_tree_keep(*dev, *b, path.long(), kept)
    with pytest.raises(mq.MqError):
        mq.kv8_tree_keep(*dev, *b, torch.zeros((1, 2000), dtype=torch.int32, device="cuda"), kept)
