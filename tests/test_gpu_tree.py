"""Trees of drafted tokens on an MI355X: masks and positions exact, attention
under any mask within the bound of each row (``oracle.fp8.kv8_attention_rows``):
both forms, every page size and head layout, masks that leave rows empty, bits
behind the last token, NaN codes in branches that a row does not see."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import drafts as od
from oracle import fp8 as o8
from tests.draft_util import offsets, random_trees, words_of
from tests.fp8_util import codes_tensor, half_tensor
from tests.gpu_util import announce, host
from tests.kv8_util import paged, put, up

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# masks and positions
# ---------------------------------------------------------------------------

def _check_mask(news, totals, parents, pad=0, most=None):
    import torch
    most = most or max(max(news), 1)
    width = -(-most // 32)
    cu, T = offsets(news), sum(news) + pad
    announce(f"kv8_tree_mask new={news[:5]} most={most}")
    parents = np.concatenate([parents, np.zeros(pad, np.int32)]).astype(np.int32)
    mask = torch.full((T, width), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    mq.kv8_tree_mask(up(parents), up(cu), up(np.array(totals, np.int32)), most, mask=mask, positions=pos)
    want, where = od.tree_ref(parents[:sum(news)], cu, totals, width)
    assert np.array_equal(host(mask)[:sum(news)], want) and np.array_equal(host(pos)[:sum(news)], where)
    assert np.all(host(mask)[sum(news):] == 77) and np.all(host(pos)[sum(news):] == 77)


@pytest.mark.parametrize("news", [[1], [8], [32, 33, 31], [64, 1, 0, 65], [200, 7], [1024], [1023, 1, 1024]])
def test_masks(news):
    rng = np.random.default_rng(sum(news))
    totals = [n + int(t) for n, t in zip(news, rng.integers(0, 3000, len(news)))]
    _check_mask(news, totals, random_trees(rng, news))
    _check_mask(news, totals, random_trees(rng, news, back=1000, loose=0.1), pad=3)
    _check_mask(news, totals, np.concatenate([np.arange(-1, n - 1) for n in news]), most=min(max(news) + 40, 1024))


def test_masks_of_bad_parents():
    """Parents that are none before their node hang on the context: own number, later ones, far ones."""
    _check_mask([9, 3], [20, 1], np.array([0, 1, 0, 9, 2 ** 31 - 1, -2 ** 31, 4, -7, 7, 5, 0, 1]))


def test_masks_of_many_sequences():
    rng = np.random.default_rng(1)
    news = [int(n) for n in rng.integers(0, 40, 300)]
    _check_mask(news, [n + 5 for n in news], random_trees(rng, news))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attend(tq, tree, cache, table, cu, lens, what, scale=None, most=None):
    import torch
    announce(f"kv8_tree_attention {what} {tq.dtype} q={tuple(tq.shape)} new={np.diff(cu)[:5].tolist()} total={list(lens)[:5]}")
    out = torch.full(tq.shape, 7.0, dtype=tq.dtype, device="cuda")
    mq.kv8_tree_attention(tq, up(tree), codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3]),
                          up(table), up(np.asarray(cu, np.int32)), up(np.asarray(lens, np.int32)),
                          max_q_len=most or max(1, int(np.max(np.diff(cu)))), softmax_scale=scale, out=out)
    return host(out.float()).astype(np.float64)


def check(rng, news, totals, Hkv, G, D, page, half, what, tree=None, qamp=1.0, width=None, pad=0, cache=None, table=None,
          scale=None, most=None, vexp=None):
    if cache is None:
        cache, table = paged(rng, [max(t, 1) for t in totals], Hkv, page, D, width)
    if vexp:
        cache[3][:] = np.exp2(rng.integers(*vexp, cache[3].shape))
    cu = offsets(news)
    T = int(cu[-1]) + pad
    if tree is None:
        tree = words_of(random_trees(rng, news), news, totals)
    tree = np.concatenate([tree, np.zeros((T - len(tree), tree.shape[1]), np.int32)])
    tq, qf = half_tensor(rng.standard_normal((T, Hkv * G, D)) * qamp, half)
    scale = D ** -0.5 if scale is None else scale
    got = attend(tq, tree, cache, table, cu, totals, what, scale, most)
    o64, bound = o8.kv8_attention_rows(qf, *cache, table, cu, totals, scale, half, tree=tree)
    none = np.isnan(o64)
    assert np.all(got[none] == 7.0), f"{what}: rows of no sequence changed"
    over = np.where(none, 0.0, np.abs(got - o64) / bound)
    assert not np.isnan(over).any(), f"{what}: NaN in row {np.argwhere(np.isnan(over))[0].tolist()}"
    assert np.all(over <= 1.0), f"{what}: worst err/bound {over.max():.3g} at {np.unravel_index(over.argmax(), over.shape)}"
    return got


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_lengths(page, D, half):
    rng = np.random.default_rng(page * D)
    check(rng, [8] * 9, [8, 9, 16, 63, 64, 65, 71, 72, 300], 2, 4, D, page, half, "eight drafts")
    check(rng, [1, 1, 1, 1], [1, 2, 64, 129], 2, 4, D, page, half, "single tokens")
    check(rng, [64, 40, 63], [64, 300, 129], 2, 4, D, page, half, "full trees")
    check(rng, [90, 3], [200, 700], 2, 3, D, page, half, "wide table", width=65536 // page)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16, 32])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_head_layouts(Hkv, G):
    rng = np.random.default_rng(G * 10 + Hkv)
    check(rng, [5, 26, 1], [300, 26, 77], Hkv, G, 128, 64, "bf16", "head layouts")


@pytest.mark.parametrize("news,G", [([2], 1), ([3, 16], 4), ([13], 8), ([17, 31, 32], 2), ([33, 64, 7], 7), ([100, 128], 4),
                                    ([150], 8), ([256, 255], 2), ([400], 5), ([1024], 1), ([700, 1000], 2)])
@pytest.mark.parametrize("context", [0, 37, 1500])
def test_tree_sizes(news, G, context):
    rng = np.random.default_rng(sum(news) + context)
    check(rng, news, [n + context + 11 * i for i, n in enumerate(news)], 2, G, 128, 32, "bf16", "tree sizes")
    check(rng, news, [n + context + 64 * i for i, n in enumerate(news)], 1, G, 64, 64, "fp16", "tree sizes")


def test_long_context():
    rng = np.random.default_rng(2)
    check(rng, [64, 20], [9000, 5000], 1, 4, 128, 64, "bf16", "long")
    check(rng, [8], [9000], 2, 4, 128, 16, "fp16", "long, few")
    check(rng, [200], [6000], 1, 4, 64, 32, "bf16", "long, many", qamp=4.0)


@pytest.mark.parametrize("news,totals,width", [([8, 5], [70, 40], None), ([70, 64], [300, 64], None), ([90, 30], [200, 30], 4096)])
def test_any_bits(news, totals, width):
    """Bits that no tree has: rows that see nothing but the context, later tokens,
    not themselves; bits behind the last token; words more than needed."""
    rng = np.random.default_rng(3)
    for words in (-(-max(news) // 32), -(-max(news) // 32) + 2):
        tree = rng.integers(-2 ** 31, 2 ** 31, (sum(news), words), dtype=np.int64).astype(np.int32)
        tree[::3] = 0
        tree[1::7] = -1
        check(rng, news, totals, 2, 4, 128, 16, "bf16", "any bits", tree=tree, width=width)


@pytest.mark.parametrize("width", [None, 4096])
def test_rows_that_see_nothing(width):
    """No context and no bits: 0. More new tokens than cached ones: the first are none."""
    rng = np.random.default_rng(4)
    for news, totals in (([6, 4], [6, 3]), ([100, 40], [100, 20]), ([90, 2], [0, 1])):
        tree = words_of(random_trees(rng, news), news, totals)
        tree[::2] = 0
        got = check(rng, news, totals, 2, 2, 64, 16, "fp16", "empty rows", tree=tree, pad=2, width=width)
        if totals[0] == news[0]:
            assert np.all(got[0:news[0]:2] == 0)


@pytest.mark.parametrize("width", [None, 4096])
@pytest.mark.parametrize("D", [64, 128])
def test_more_new_tokens_than_cached(D, width):
    """The first of the new tokens then have no place, and no row sees them."""
    rng = np.random.default_rng(16)
    news, totals = [20, 9, 70, 70, 1], [12, 0, 30, 70, 0]
    for tree in (words_of(random_trees(rng, news), news, totals, 4),
                 rng.integers(-2 ** 31, 2 ** 31, (170, 4), dtype=np.int64).astype(np.int32)):
        got = check(rng, news, totals, 2, 4, D, 16, "bf16", "more new than cached", width=width, tree=tree, most=100, pad=3)
        assert not got[20:29].any() and not got[169:170].any()


def test_unknown_pages():
    rng = np.random.default_rng(5)
    for news, G, width in (([4, 2], 4, None), ([90, 40], 2, 4096)):
        cache, table = paged(rng, [150, 75], 2, 16, 128, width)
        table[0, 2], table[0, 8], table[1, 4] = -1, 2 ** 31 - 1, -7
        check(rng, news, [150, 75], 2, G, 128, 16, "bf16", "unknown pages", cache=cache, table=table)
        check(rng, news, [150, 75], 2, G, 128, 16, "bf16", "narrow table", cache=cache, table=table[:, :6].copy())


@pytest.mark.parametrize("news,totals,width", [([8], [500], None), ([64], [1500], None), ([150, 20], [600, 90], 4096)])
def test_peaked_scores_and_wide_scales(news, totals, width):
    rng = np.random.default_rng(6)
    check(rng, news, totals, 2, 4, 128, 32, "bf16", "peaked", qamp=12.0, width=width)
    check(rng, news, totals, 2, 4, 128, 16, "fp16", "wide scales", vexp=(-30, 6), width=width)
    check(rng, news, totals, 1, 4, 64, 16, "fp16", "no scale", scale=0.0, width=width)


@pytest.mark.parametrize("news,totals,G,width", [([8], [100], 4, None), ([20], [20], 2, None), ([64, 9], [200, 70], 4, None),
                                                 ([100, 64], [333, 128], 4, 4096), ([300], [300], 2, 4096)])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_stays_in_its_branch(news, totals, G, width, D):
    """NaN codes of K and V in some drafts: rows that do not see them are what they
    are without, rows that do get NaN (K: the whole row, V: its dimensions)."""
    rng = np.random.default_rng(sum(news) + D)
    Hkv, page = 2, 16
    cache, table = paged(rng, totals, Hkv, page, D, width)
    tree = words_of(random_trees(rng, news), news, totals)
    cu = offsets(news)
    clean = tuple(c.copy() for c in cache)
    hit_k, hit_v = np.zeros((sum(news), Hkv), bool), np.zeros((sum(news), Hkv, D), bool)
    for b, (n, total) in enumerate(zip(news, totals)):
        for j in rng.choice(n, max(1, n // 6), replace=False):
            start, sees = total - n, (tree[cu[b]:cu[b + 1], j // 32] >> (j % 32)) & 1 == 1
            head, d, kind = int(rng.integers(Hkv)), int(rng.integers(D)), int(rng.integers(2))
            p, t = table[b, (start + j) // page], (start + j) % page
            if kind:
                cache[0][p, head, t, d] = rng.choice([0x7F, 0xFF])
                clean[0][p, head, t, d] = 0
                hit_k[cu[b]:cu[b + 1], head] |= sees
            else:
                cache[1][p, head, d, t] = rng.choice([0x7F, 0xFF])
                clean[1][p, head, d, t] = 0
                hit_v[cu[b]:cu[b + 1], head, d] |= sees
    tq, qf = half_tensor(rng.standard_normal((sum(news), Hkv * G, D)), "bf16")
    got = attend(tq, tree, cache, table, cu, totals, "nan", D ** -0.5)
    o64, bound = o8.kv8_attention_rows(qf, *clean, table, cu, totals, D ** -0.5, "bf16", tree=tree)
    nan = np.repeat(hit_k[:, :, None] | hit_v, G, axis=1)
    assert np.isnan(got[nan]).all(), "a NaN was lost"
    # without its V code a row's other dimensions keep their weights, so the bound holds there
    keep = ~np.repeat(hit_k, G, axis=1)[:, :, None] & ~nan
    over = np.where(keep, np.abs(got - o64) / bound, 0.0)
    assert not np.isnan(over).any(), "a NaN left its branch"
    assert np.all(over <= 1.0), f"worst err/bound {over.max():.3g}"


def test_nan_behind_the_last_token_counts_for_nothing():
    """paged() fills what no token holds with NaN codes; so do pages of no sequence."""
    rng = np.random.default_rng(8)
    cache, table = paged(rng, [77, 100], 2, 64, 128)
    for b, t in ((0, 77), (1, 100)):
        put(cache, table, b, t, k=np.full(128, 0x7F, np.uint8), v=np.full(128, 0xFF, np.uint8))
    check(rng, [30, 13], [77, 100], 2, 4, 128, 64, "bf16", "behind the last", cache=cache, table=table)


def test_agrees_with_causal_attention():
    """A chain's mask sees what causal attention sees: both within a row's bounds."""
    rng = np.random.default_rng(9)
    for news, totals in (([5, 20], [400, 33]), ([128], [900])):
        cache, table = paged(rng, totals, 2, 32, 128)
        cu = offsets(news)
        tree = words_of(np.concatenate([np.arange(-1, n - 1) for n in news]), news, totals)
        tq, qf = half_tensor(rng.standard_normal((sum(news), 8, 128)), "fp16")
        got = attend(tq, tree, cache, table, cu, totals, "chain", 0.1)
        dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
        causal = host(mq.kv8_attention(tq, *dev, up(table), up(cu), up(np.array(totals, np.int32)), max_q_len=max(news),
                                       softmax_scale=0.1).float()).astype(np.float64)
        _, bound = o8.kv8_attention_rows(qf, *cache, table, cu, totals, 0.1, "fp16", tree=tree)
        assert np.all(np.abs(got - causal) <= 2 * bound)


@pytest.mark.parametrize("page,width", [(16, None), (64, 512)])
def test_many_sequences(page, width):
    """More sequences than a wavefront has lanes, so that shares are counted in
    several steps: some without new tokens, a few large trees over long contexts."""
    rng = np.random.default_rng(12)
    news = [int(n) for n in rng.integers(0, 30, 150)]
    news[0], news[70], news[149] = 0, 300, 200
    totals = [n + int(t) for n, t in zip(news, rng.integers(0, 60, 150))]
    for b in (3, 64, 70, 149):
        totals[b] += 2500
    check(rng, news, totals, 1, 4, 64, page, "bf16", "many sequences", pad=2, width=width)
    check(rng, news[60:130], totals[60:130], 2, 3, 128, page, "fp16", "many sequences", width=width)


def test_pages_past_4_gb():
    """The same step on pages at the end of a cache of 4.8 GB and on a small one."""
    import torch
    rng = np.random.default_rng(13)
    H, page, D, news, totals = 8, 128, 128, [40, 3], [300, 200]
    cu, tree = offsets(news), words_of(random_trees(rng, news), news, totals)
    T, used, P = 43, 5, 36700
    qkv, _ = half_tensor(rng.standard_normal((T, 32 + 2 * H, D)), "bf16")
    angles = rng.uniform(0, 6, (400, 64))
    cs = up(np.concatenate([np.cos(angles), np.sin(angles)], 1).astype(np.float32))
    path, kept = up(np.array([[0, 3, 9, 20], [0, 2, -1, -1]], np.int32)), up(np.array([4, 2], np.int32))
    codes = [torch.from_numpy(rng.integers(0, 120, (used, H, page, D)).astype(np.uint8)).cuda() for _ in "kv"]
    results = []
    for pages, first in ((used, 0), (P, P - used)):
        dev = [torch.zeros((pages, H, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
               torch.zeros((pages, H, D, page), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
               torch.full((pages, H), 2.0 ** -6, device="cuda"), torch.full((pages, H), 2.0 ** -6, device="cuda")]
        dev[0].view(torch.uint8)[first:] = codes[0]
        dev[1].view(torch.uint8)[first:] = codes[1].transpose(2, 3)
        table = up((np.array([[0, 1, 2], [3, 4, 2 ** 20]]) + first).astype(np.int32))
        b = table, up(cu), up(np.array(totals, np.int32))
        announce(f"drafts on pages from {first} on")
        q, k, v = qkv.split([32, H, H], 1)
        q = mq.kv8_rope_append(q, k, v, *dev, *b, 40, cs)
        o = mq.kv8_tree_attention(q, up(tree), *dev, *b, max_q_len=40)
        mq.kv8_tree_keep(*dev, *b, path, kept)
        results.append([q, o] + [t.view(torch.uint8)[first:].clone() for t in dev])
        assert not dev[0].view(torch.uint8)[:first].any() and not dev[1].view(torch.uint8)[:first].any()
        del dev
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_strided_queries_and_workspace():
    import torch
    rng = np.random.default_rng(10)
    news, totals = [26, 9], [700, 2000]
    cache, table = paged(rng, totals, 2, 32, 128)
    cu, tree = offsets(news), words_of(random_trees(rng, news), news, totals)
    fused, _ = half_tensor(rng.standard_normal((35, 12, 128)), "bf16")
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    b = up(table), up(cu), up(np.array(totals, np.int32))
    need = mq.kv8_tree_attention_workspace_bytes(35, 2, 8, 2, 128, 32, table.shape[1], 26)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
    announce("kv8_tree_attention strided")
    one = mq.kv8_tree_attention(fused[:, 2:10], up(tree), *dev, *b, max_q_len=26, workspace=ws)
    two = mq.kv8_tree_attention(fused[:, 2:10].contiguous(), up(tree), *dev, *b, max_q_len=26)
    assert torch.equal(one, two) and not torch.isnan(one.float()).any()
    again = mq.kv8_tree_attention(fused[:, 2:10], up(tree), *dev, *b, max_q_len=26, workspace=ws)
    assert torch.equal(one, again)


def test_refusals_of_the_wrappers():
    import torch
    rng = np.random.default_rng(11)
    cache, table = paged(rng, [20], 2, 16, 64)
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    b = up(table), up(np.array([0, 4], np.int32)), up(np.array([20], np.int32))
    q = torch.zeros((4, 4, 64), dtype=torch.float16, device="cuda")
    tree = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    mq.kv8_tree_attention(q, tree, *dev, *b, 4)
    with pytest.raises(TypeError):
        mq.kv8_tree_attention(q, tree.long(), *dev, *b, 4)
    with pytest.raises(ValueError):
        mq.kv8_tree_attention(q, tree[:3], *dev, *b, 4)
    with pytest.raises(mq.MqError):
        mq.kv8_tree_attention(q, tree, *dev, *b, 40)
    with pytest.raises(mq.MqError):
        mq.kv8_tree_attention(q, torch.zeros((4, 64), dtype=torch.int32, device="cuda"), *dev, *b, 2000)
    with pytest.raises(ValueError):
        mq.kv8_tree_mask(tree[:, 0].contiguous(), b[1], b[2], 2000)
    with pytest.raises(ValueError):
        mq.kv8_tree_mask(tree[:, 0].contiguous(), b[1], b[2][:0], 4)
    with pytest.raises(ValueError):
        mq.kv8_tree_mask(tree[:, 0].contiguous(), b[1], b[2], 4, positions=b[2])
