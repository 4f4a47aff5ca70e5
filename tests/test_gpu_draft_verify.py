"""Verification of drafted tokens on an MI355X: kept nodes, paths and the drawn
token equal the oracle's, for trees and chains, random rows and rows of dyadic
probabilities whose borders the uniform numbers hit exactly."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import drafts as od
from tests.draft_util import offsets, random_trees, up
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu


def check(probs, tokens, uniform, news, what, parents=None, draft=None, most=None, pad=0):
    import torch
    cu, most = offsets(news), most or max(max(news), 1)
    announce(f"draft_verify {what} probs={probs.shape} new={list(news)[:5]}")

    def padded(a):
        return None if a is None else up(np.concatenate([a, np.ones((pad, *a.shape[1:]), a.dtype)]))

    ws = torch.full((mq.draft_verify_workspace_bytes(len(news), probs.shape[1], most),), 255, dtype=torch.uint8, device="cuda")
    got = mq.draft_verify(padded(probs), padded(tokens), padded(uniform), up(cu), most, parents=padded(parents),
                          draft_probs=padded(draft), workspace=ws)
    with np.errstate(invalid="ignore"):
        want = od.verify_ref(probs, tokens, uniform, cu, most, parents, draft)
    for name, g, w in zip(("kept", "path", "next"), got, want):
        assert np.array_equal(host(g), w), f"{what}: {name} {host(g).tolist()[:6]} instead of {w.tolist()[:6]}"
    return want


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def tree_case(rng, news, V, sharp=3.0, loose=0.0):
    """Siblings are the likeliest tokens of their parent's row, now and then the same twice."""
    parents = random_trees(rng, news, loose=loose)
    probs = softmax(sharp * rng.standard_normal((sum(news), V)))
    tokens, cu = np.zeros(sum(news), np.int32), offsets(news)
    for b, n in enumerate(news):
        for j in range(1, n):
            up_ = max(parents[cu[b] + j], 0)
            older = int(np.sum(parents[cu[b] + 1:cu[b] + j] == up_))
            if rng.random() < 0.1:
                older = max(older - 1, 0)
            row = probs[cu[b] + up_]
            tokens[cu[b] + j] = np.argsort(-row, kind="stable")[min(older, V - 1)]
    return probs, tokens, rng.random(sum(news)).astype(np.float32), parents


@pytest.mark.parametrize("V", [1, 2, 63, 64, 1000, 4095, 4096, 4097, 32000, 50001])
@pytest.mark.parametrize("news", [[1], [8, 3], [1, 0, 26, 5, 12, 12, 12]])
def test_trees(V, news):
    rng = np.random.default_rng(V + sum(news))
    for rep in range(3):
        probs, tokens, uniform, parents = tree_case(rng, news, V)
        kept, _, _ = check(probs, tokens, uniform, news, "trees", parents=parents, pad=rep)


@pytest.mark.parametrize("V", [2, 64, 1000, 4097, 32000])
@pytest.mark.parametrize("given", [True, False])
def test_chains(V, given):
    rng = np.random.default_rng(V)
    news = [6, 1, 4, 0, 9, 6, 6, 6, 2]
    for rep in range(4):
        logits = 2 * rng.standard_normal((sum(news), V))
        probs, draft = softmax(logits), softmax(logits + 0.7 * rng.standard_normal(logits.shape))
        tokens, cu = np.zeros(sum(news), np.int32), offsets(news)
        for b, n in enumerate(news):
            for j in range(1, n):
                row = draft[cu[b] + j - 1].astype(np.float64)
                tokens[cu[b] + j] = rng.choice(V, p=row / row.sum())
        check(probs, tokens, rng.random(sum(news)).astype(np.float32), news, "chains", draft=draft if given else None,
              most=9 + rep)


@pytest.mark.parametrize("V", [65536, 65537, 70001, 140000, 300003])
def test_long_rows(V):
    """Rows of more pieces than one workgroup takes, aligned and not."""
    rng = np.random.default_rng(V)
    news = [5, 1, 0, 8]
    for rep in range(2):
        probs, tokens, uniform, parents = tree_case(rng, news, V, sharp=2.0 + 2 * rep)
        check(probs, tokens, uniform, news, "long rows", parents=parents, pad=rep)
        draft = softmax(np.log(probs + 1e-12) + 0.7 * rng.standard_normal(probs.shape))
        check(probs, tokens, uniform, news, "long rows, chains", draft=draft)
    flat = np.full((6, V), 1 / V, np.float32)
    for u in (0.0, 0.25, 0.75, 0.99999994):
        check(flat, np.array([0, 3, 5, V - 1, 0, 1], np.int32), np.full(6, u, np.float32), [4, 2], "flat")


@pytest.mark.parametrize("V", [1000, 66000])
def test_many_sequences(V):
    rng = np.random.default_rng(V)
    news = [int(n) for n in rng.integers(0, 3, 300)]
    probs, tokens, uniform, parents = tree_case(rng, news, V)
    check(probs, tokens, uniform, news, "many sequences", parents=parents)


def test_large_trees():
    rng = np.random.default_rng(1)
    for news in ([64, 200], [1024, 65]):
        probs, tokens, uniform, parents = tree_case(rng, news, 300, sharp=2.0, loose=0.02)
        check(probs, tokens, uniform, news, "large trees", parents=parents, most=1024)
    # many children of one node: those of several wavefront steps, all rejected or not
    n = 300
    parents = np.zeros(n, np.int32) - (np.arange(n) == 0)
    probs = np.full((n, 512), 1 / 512, np.float32)
    for at in (0.999, 0.5, 0.001):
        u = np.full(n, at, np.float32)
        check(probs, rng.permutation(512)[:n].astype(np.int32), u, [n], "wide", parents=parents)
        check(probs, np.full(n, 7, np.int32), u, [n], "one token only", parents=parents)


def test_exact_borders():
    """Probabilities of n/64 and uniform numbers of k/64: every comparison is exact,
    equality among them; zeros are never drawn."""
    rng = np.random.default_rng(2)
    for V in (8, 70, 5000):
        for rep in range(40):
            news = [5, 2, 3]
            parts = np.zeros((sum(news), V))
            for r in range(sum(news)):
                at = rng.integers(0, V, 64 if rep % 2 else 4)
                np.add.at(parts[r], at, 64 // len(at))
            probs = (parts / 64).astype(np.float32)
            tokens = np.array([rng.choice(np.flatnonzero(parts[rng.integers(0, sum(news))])) for _ in range(sum(news))], np.int32)
            uniform = (rng.integers(0, 64, sum(news)) / 64).astype(np.float32)
            draft = np.roll(probs, 1, axis=1) if rep % 4 == 3 else None
            parents = None if rep % 4 else random_trees(rng, news)
            check(probs, tokens, uniform, news, "borders", parents=parents, draft=draft)


def test_greedy_rows():
    """One-hot rows: the longest path of the tree that the target would have taken."""
    probs = np.zeros((6, 100), np.float32)
    probs[np.arange(6), [5, 9, 7, 1, 2, 3]] = 1
    #  0 -> 1 (4), 2 (5);  2 -> 3 (8), 4 (7);  4 -> 5 (0)
    parents, tokens = np.array([-1, 0, 0, 2, 2, 4], np.int32), np.array([50, 4, 5, 8, 7, 0], np.int32)
    for u in (0.0, 0.5, 0.99999994):
        want = check(probs, tokens, np.full(6, u, np.float32), [6], "greedy", parents=parents)
        assert want[0].tolist() == [3] and want[1][0, :3].tolist() == [0, 2, 4] and want[2].tolist() == [2]


def test_odd_rows():
    """Rows without mass, NaN, negative and infinite values, tokens outside the
    vocabulary, uniform numbers of 0 and just below 1."""
    rng = np.random.default_rng(3)
    V, news = 5000, [3, 3, 3, 3, 3]
    base = softmax(rng.standard_normal((15, V)))
    for kind in range(4):
        probs = base.copy()
        tokens = rng.integers(0, V, 15).astype(np.int32)
        if kind == 0:
            probs[:6] = 0
        elif kind == 1:
            probs[:, ::7] = np.nan
            probs[3:6] = np.nan
        elif kind == 2:
            probs[:, ::5] *= -1
        else:
            tokens[1::3] = [-1, V, 2 ** 31 - 1, -2 ** 31, V + 7]
        for u in (0.0, 0.99999994, 0.3):
            check(probs, tokens, np.full(15, u, np.float32), news, f"odd {kind}")
            check(probs, tokens, np.full(15, u, np.float32), news, f"odd {kind}, draft", draft=base)
    import torch
    probs = torch.from_numpy(base).cuda()
    probs[0, 17] = float("inf")
    got = mq.draft_verify(probs, up(tokens), up(np.full(15, 0.5, np.float32)), up(offsets(news)), 3)
    assert all(0 <= int(t) < V for t in got[2].cpu())  # (which one is not defined)


def test_tokens_without_mass_are_not_taken():
    """Siblings whose probabilities add up to more than 1 by rounding, then one of
    probability 0 and one rejected before: neither is taken."""
    V = 50
    probs = np.zeros((5, V), np.float32)
    probs[:, 3], probs[:, 4] = 0.6, np.float32(0.4) + np.float32(2.0 ** -20)
    parents = np.array([-1, 0, 0, 0, 0], np.int32)
    tokens = np.array([9, 3, 4, 7, 3], np.int32)
    u = np.array([0.5, 0.999, 0.99999994, 0.5, 0.5], np.float32)
    u[2] = 1.5  # (no number of [0, 1): both siblings with mass are rejected)
    want = check(probs, tokens, u, [5], "no mass", parents=parents)
    assert want[0].tolist() == [1] and want[2].tolist() == [3]  # nothing is left: the row itself
    draft = probs.copy()
    draft[:, ::5] = np.nan
    draft[:, 1::5] = -1
    for x in (3, 5, 6):
        check(probs, np.full(5, x, np.int32), np.full(5, 0.25, np.float32), [5], "odd drafts", draft=draft)


def test_rejected_token_is_not_drawn():
    """All but a rejected token have next to nothing: it still is not drawn again."""
    V = 9000
    probs = np.full((2, V), 1e-12, np.float32)
    probs[:, 4321] = 1 - 1e-6
    u = np.array([0.7, 0.99999994], np.float32)
    want = check(probs, np.array([0, 4321], np.int32), u, [2], "rejected")
    assert want[0].tolist() == [1] and want[2][0] != 4321


def test_rows_past_2_31_values():
    """The same drafts in the last rows of 9.4 GB of probabilities and in a small tensor."""
    import torch
    rng = np.random.default_rng(14)
    V, T, news = 2 ** 24, 140, [4, 3]
    first = T - sum(news)
    rows = torch.zeros((sum(news), V), device="cuda")
    at = rng.integers(0, V, (sum(news), 50))
    rows.scatter_(1, up(at), up(softmax(rng.standard_normal(at.shape))))
    tokens, uniform = np.zeros(T, np.int32), rng.random(T).astype(np.float32)
    for j in (1, 2, 3, 5, 6):
        tokens[first + j] = at[j - 1 if j != 6 else 4][j]
    parents = np.zeros(T, np.int32)
    parents[first:] = [-1, 0, 1, 2, -1, 0, 0]
    uniform[first + 1:first + 3] = 0  # these two are taken: their tokens have some mass
    probs = torch.zeros((T, V), device="cuda")
    probs[first:] = rows
    announce("draft_verify 140 rows of 2^24")
    got = mq.draft_verify(probs, up(tokens), up(uniform), up(np.array([first, first + 4, T], np.int32)), 4, parents=up(parents))
    want = mq.draft_verify(rows, up(tokens[first:]), up(uniform[first:]), up(offsets(news)), 4, parents=up(parents[first:]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert host(got[0]).max() > 1 and host(got[2]).min() >= 0
    assert all(int(t) in at[p] for t, p in zip(host(got[2]), [int(host(got[1])[0][host(got[0])[0] - 1]), 4 + int(host(got[1])[1][host(got[0])[1] - 1])]))


def test_workspace_and_outputs_of_the_caller():
    import torch
    rng = np.random.default_rng(4)
    news = [8, 5]
    probs, tokens, uniform, parents = tree_case(rng, news, 6000)
    args = up(probs), up(tokens), up(uniform), up(offsets(news))
    a = mq.draft_verify(*args, 8, parents=up(parents))
    mine = [torch.full(s, 9, dtype=torch.int32, device="cuda") for s in ((2,), (2, 8), (2,))]
    b = mq.draft_verify(*args, 8, parents=up(parents), kept=mine[0], path=mine[1], next_token=mine[2])
    assert all(torch.equal(x, y) and y.data_ptr() == z.data_ptr() for x, y, z in zip(a, b, mine))
    with pytest.raises(ValueError):
        mq.draft_verify(*args, 8, parents=up(parents), draft_probs=args[0])
    with pytest.raises(ValueError):
        mq.draft_verify(*args, 8, path=mine[1][:, :7])
    with pytest.raises(TypeError):
        mq.draft_verify(args[0].half(), *args[1:], 8)
    long = torch.full((13, 200001), 1 / 200001, device="cuda")
    with pytest.raises(mq.MqError):
        mq.draft_verify(long, *args[1:], 8, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    empty = mq.draft_verify(args[0][:0], args[1][:0], args[2][:0], up(np.zeros(3, np.int32)), 4)
    assert empty[0].tolist() == [0, 0] and empty[1].tolist() == [[-1] * 4] * 2 and empty[2].tolist() == [-1, -1]
