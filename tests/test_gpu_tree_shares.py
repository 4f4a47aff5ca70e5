"""Attention of drafted tokens where the keys are shared out on the GPU by the
sequences' lengths: more row tiles than the workspace has parts."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.draft_util import offsets, random_trees, words_of
from tests.fp8_util import codes_tensor, half_tensor
from tests.gpu_util import announce, host
from tests.kv8_util import paged, up

pytestmark = pytest.mark.gpu

GUARD = 4096


def guarded(rng, news, totals, Hkv, G, D, page, half, width=None):
    """Rows within their bounds, nothing written behind the workspace."""
    import torch
    cache, table = paged(rng, [max(t, 1) for t in totals], Hkv, page, D, width)
    cu, T, most = offsets(news), sum(news), max(news)
    tree = words_of(random_trees(rng, news), news, totals)
    tq, qf = half_tensor(rng.standard_normal((T, Hkv * G, D)), half)
    need = mq.kv8_tree_attention_workspace_bytes(T, len(news), Hkv * G, Hkv, D, page, table.shape[1], most)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
    announce(f"kv8_tree_attention of {len(news)} trees, {Hkv} x {G} heads of {D}, workspace {need}")
    got = host(mq.kv8_tree_attention(tq, up(tree), codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3]),
                                     up(table), up(cu), up(np.array(totals, np.int32)), most, workspace=ws[:need]).float())
    assert torch.all(ws[need:] == 255)
    o64, bound = o8.kv8_attention_rows(qf, *cache, table, cu, totals, D ** -0.5, half, tree=tree)
    over = np.abs(got - o64) / bound
    assert np.all(over <= 1.0), f"worst err/bound {np.nanmax(over):.3g}, {np.isnan(over).sum()} NaN"


@pytest.mark.parametrize("seqs,Hkv,G,D,page", [(70, 8, 16, 64, 64), (40, 8, 16, 128, 32), (200, 5, 8, 64, 128)])
def test_many_row_tiles(seqs, Hkv, G, D, page):
    """Most sequences in one share, the long ones in several."""
    rng = np.random.default_rng(seqs)
    news = [int(n) for n in rng.integers(17, 34, seqs)]
    totals = [n + int(t) for n, t in zip(news, rng.integers(0, 200, seqs))]
    for b in (0, seqs // 2, seqs - 1):
        totals[b] += 3000
    guarded(rng, news, totals, Hkv, G, D, page, "bf16")
