"""Attention of drafted tokens where the keys are shared out on the GPU by the
sequences' lengths: more row tiles than the workspace has parts, kv heads that do
not divide the shares, shares of more tiles than one batch of page numbers and
scales holds, one captured call over changing lengths."""

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
    sizes = T, len(news), Hkv * G, Hkv, D, page, table.shape[1], most
    need = mq.kv8_tree_attention_workspace_bytes(*sizes)
    assert mq.kv8_tree_attention_form(*sizes) == "prompt" and need > 0
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


@pytest.mark.parametrize("Hkv,G", [(3, 3), (5, 4), (7, 2), (8, 4), (12, 2), (100, 1)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_head_layouts(Hkv, G, D, page):
    rng = np.random.default_rng(Hkv + D)
    guarded(rng, [70, 1, 90, 33], [70 + 1900, 600, 90, 33 + 170], Hkv, G, D, page, "fp16", width=65536 // page)


def mean_tiles(news, totals, Hkv, G):
    """Tiles of 64 keys a share has at least on average: 256 shares, or two a row tile."""
    rows = [-(-n * G // 256) * Hkv for n in news]
    return sum(r * -(-t // 64) for r, t in zip(rows, totals)) / max(256, 2 * sum(rows))


@pytest.mark.parametrize("news,totals,Hkv,G,D,page,half", [
    ([256, 130, 64], [9000, 8000, 5000], 8, 4, 64, 32, "bf16"),
    ([200, 90, 37], [9000, 7000, 300], 5, 7, 128, 64, "fp16"),
    ([64, 50, 9], [11000, 300, 9000], 12, 8, 128, 128, "bf16"),
])
def test_long_shares(news, totals, Hkv, G, D, page, half):
    """Page numbers and scales come 16 tiles at a time: shares of two batches and more."""
    assert mean_tiles(news, totals, Hkv, G) > 20
    guarded(np.random.default_rng(Hkv), news, totals, Hkv, G, D, page, half)


def _padded(rng, seqs, most, longest):
    """A batch of some sequence lengths: whoever has fewer new tokens leaves rows at the end."""
    news = [int(n) for n in rng.integers(0, most + 1, seqs)]
    totals = [n + int(longest * rng.random() ** 3) for n in news]
    return news, totals


@pytest.mark.parametrize("seqs,Hkv,G,D,page", [(3, 8, 4, 128, 32), (8, 8, 4, 64, 64), (70, 3, 2, 64, 16)])
def test_captured_call_over_changing_lengths(seqs, Hkv, G, D, page):
    """One graph, replayed over batches of other lengths, trees and pages: the bits of
    the eager calls, rows of no sequence left alone."""
    import torch
    rng = np.random.default_rng(seqs)
    most, longest, T = 70, 4000, 70 * seqs
    width = -(-(longest + most) // page)
    steps = [_padded(rng, seqs, most, longest) for _ in range(3)]
    steps.append(([0] * (seqs - 1) + [most], [5] * (seqs - 1) + [longest + most]))  # one sequence alone, the longest there is
    steps.append(([most] * seqs, [most] * seqs))
    steps.append(([0] * seqs, [9] * seqs))
    pool = -(-max(sum(-(-t // page) for t in totals) for _, totals in steps) // 8) * 8
    k = torch.from_numpy(rng.integers(0, 120, (pool, Hkv, page, D)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
    v = torch.from_numpy(rng.integers(0, 120, (pool, Hkv, D, page)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
    scales = [up(np.exp2(rng.integers(-12, -8, (pool, Hkv))).astype(np.float32)) for _ in "kv"]
    i32 = dict(dtype=torch.int32, device="cuda")
    table, cu, lens = torch.zeros((seqs, width), **i32), torch.zeros(seqs + 1, **i32), torch.zeros(seqs, **i32)
    tree = torch.zeros((T, -(-most // 32)), **i32)
    q, _ = half_tensor(rng.standard_normal((T, Hkv * G, D)), "bf16")
    out = torch.zeros((T, Hkv * G, D), dtype=torch.bfloat16, device="cuda")
    sizes = T, seqs, Hkv * G, Hkv, D, page, width, most
    assert mq.kv8_tree_attention_form(*sizes) == "prompt"
    ws = torch.full((mq.kv8_tree_attention_workspace_bytes(*sizes),), 255, dtype=torch.uint8, device="cuda")

    def call(out, ws):
        return mq.kv8_tree_attention(q, tree, k, v, *scales, table, cu, lens, most, out=out, workspace=ws)

    def enter(news, totals):
        ids, at = rng.permutation(pool), 0
        host_table = np.full((seqs, width), -1, np.int32)
        for b, t in enumerate(totals):
            n = -(-t // page)
            host_table[b, :n], at = ids[at:at + n], at + n
        words = words_of(random_trees(rng, news), news, totals, tree.shape[1])
        table.copy_(up(host_table))
        cu.copy_(up(offsets(news)))
        lens.copy_(up(np.array(totals, np.int32)))
        tree[:sum(news)] = up(words)

    announce(f"captured kv8_tree_attention of {seqs} trees")
    enter(*steps[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, ws)
    for news, totals in steps + steps[:2]:
        enter(news, totals)
        eager = call(torch.full_like(out, 7.0), None)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), (news[:5], totals[:5])
        assert not torch.isnan(eager).any() and torch.all(eager[sum(news):] == 7.0)
