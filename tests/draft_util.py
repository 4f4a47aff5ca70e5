"""Batches of drafted tokens for the tests of the operators that take them."""

import numpy as np

from oracle import drafts as od
from tests.kv8_util import paged, up


def offsets(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


def random_trees(rng, news, back=6, loose=0.0):
    """Parents in each sequence's own numbers; `loose`: how many nodes but the
    first hang on the context too."""
    out = []
    for n in news:
        for j in range(n):
            p = max(0, j - 1 - int(rng.integers(0, min(j, back) + 1))) if j else -1
            out.append(-1 if rng.random() < loose else p)
    return np.array(out, np.int32)


def words_of(parents, news, totals, width=None):
    cu = offsets(news)
    width = width or -(-max(max(news), 1) // 32)
    return od.tree_ref(parents, cu, totals, width)[0]


def table_of_angles(rng, count, rot):
    """Any cosines and sines do: what stands in the table is what counts."""
    a = rng.uniform(0, 2 * np.pi, (count, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def layered(rng, layers, totals, H, page, D, width=None):
    """Caches of several layers over one table, as host arrays."""
    parts = []
    for _ in range(layers):
        cache, table = paged(np.random.default_rng(7), totals, H, page, D, width)
        P = cache[0].shape[0]
        live = (cache[0] & 0x7F) != 0x7F
        k = np.where(live, rng.integers(0, 127, cache[0].shape) | rng.integers(0, 2, cache[0].shape) << 7, cache[0])
        live = (cache[1] & 0x7F) != 0x7F
        v = np.where(live, rng.integers(0, 127, cache[1].shape) | rng.integers(0, 2, cache[1].shape) << 7, cache[1])
        parts.append((k.astype(np.uint8), v.astype(np.uint8), np.exp2(rng.integers(-12, -3, (P, H))).astype(np.float32),
                      np.exp2(rng.integers(-12, -3, (P, H))).astype(np.float32)))
    return tuple(np.stack(x) for x in zip(*parts)), table


__all__ = ["offsets", "random_trees", "words_of", "table_of_angles", "layered", "up"]
