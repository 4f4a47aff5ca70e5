"""Serving steps with drafted tokens: masks, append with rotation, attention under
the tree, verification and the cache's clean-up, as a server runs them for
several layers. Against a second cache that never saw a rejected draft; captured,
with trees and lengths that change; on two streams at once."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import drafts as od
from oracle import fp8 as o8
from tests.draft_util import offsets, random_trees, table_of_angles, up
from tests.fp8_util import codes_of, half_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, LAYERS, V, ROT = 8, 2, 64, 16, 2, 700, 64


class Server:
    """Caches of all layers over one table, and a vocabulary's head."""

    def __init__(self, seed, seqs, pages, half="bf16"):
        import torch
        rng = np.random.default_rng(seed)
        self.rng, self.half, self.seqs = rng, half, seqs
        self.dt = torch.bfloat16 if half == "bf16" else torch.float16
        P = seqs * pages + 2
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.cache = (torch.full((LAYERS, P, HKV, PAGE, D), 0x7F, **u8).view(torch.float8_e4m3fn),
                      torch.full((LAYERS, P, HKV, D, PAGE), 0x7F, **u8).view(torch.float8_e4m3fn),
                      torch.zeros((LAYERS, P, HKV), device="cuda"), torch.zeros((LAYERS, P, HKV), device="cuda"))
        self.table = up(rng.permutation(P)[:seqs * pages].reshape(seqs, pages).astype(np.int32))
        self.angles = table_of_angles(rng, pages * PAGE, ROT)
        self.cos_sin = up(self.angles)
        self.w = [half_tensor(rng.uniform(0.5, 1.5, D), half)[0] for _ in "qk"]

    def inputs(self, T):
        """Every layer's fused projection, the target's probabilities, uniform numbers, tokens."""
        import torch
        qkv = [half_tensor(self.rng.standard_normal((T, HQ + 2 * HKV, D)), self.half)[0] for _ in range(LAYERS)]
        probs = torch.softmax(torch.from_numpy(3 * self.rng.standard_normal((T, V)).astype(np.float32)).cuda(), -1)
        tokens = probs.argmax(-1).int().roll(1)  # (chains' drafts are often the likeliest)
        return qkv, probs, torch.from_numpy(self.rng.random(T).astype(np.float32)).cuda(), tokens

    def step(self, parents, cu, lens, most, qkv, probs, uniform, tokens, buf=None):
        b = buf or {}
        T = parents.shape[0]
        tree, pos = mq.kv8_tree_mask(parents, cu, lens, most, mask=b.get("mask"), positions=b.get("pos"))
        outs = []
        for i in range(LAYERS):
            q, k, v = qkv[i].split([HQ, HKV, HKV], 1)
            layer = [t[i] for t in self.cache]
            q = mq.kv8_rope_append(q, k, v, *layer, self.table, cu, lens, most, self.cos_sin, positions=pos,
                                   q_weight=self.w[0], k_weight=self.w[1], out=b.get(f"q{i}"))
            outs.append(mq.kv8_tree_attention(q, tree, *layer, self.table, cu, lens, most, out=b.get(f"o{i}"),
                                              workspace=b.get("ws")))
        kept, path, nxt = mq.draft_verify(probs, tokens, uniform, cu, most, parents=parents, kept=b.get("kept"),
                                          path=b.get("path"), next_token=b.get("next"), workspace=b.get("vws"))
        mq.kv8_tree_keep(*self.cache, self.table, cu, lens, path, kept)
        return outs, kept, path, nxt

    def buffers(self, T, most):
        import torch
        i32 = dict(dtype=torch.int32, device="cuda")
        half = dict(dtype=self.dt, device="cuda")
        b = {"mask": torch.zeros((T, -(-most // 32)), **i32), "pos": torch.zeros(T, **i32), "kept": torch.zeros(self.seqs, **i32),
             "path": torch.zeros((self.seqs, most), **i32), "next": torch.zeros(self.seqs, **i32)}
        for i in range(LAYERS):
            b[f"q{i}"], b[f"o{i}"] = torch.zeros((T, HQ, D), **half), torch.zeros((T, HQ, D), **half)
        need = mq.kv8_tree_attention_workspace_bytes(T, self.seqs, HQ, HKV, D, PAGE, self.table.shape[1], most)
        b["ws"] = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
        b["vws"] = torch.empty(mq.draft_verify_workspace_bytes(self.seqs, V, most), dtype=torch.uint8, device="cuda")
        return b


def _host(cache, layer):
    return codes_of(cache[0])[layer], codes_of(cache[1])[layer], host(cache[2])[layer], host(cache[3])[layer]


@pytest.mark.parametrize("half", ["fp16", "bf16"])
def test_steps(half):
    """Ragged steps, each operator's result against its oracle on what it got."""
    m = Server(1, 3, 10, half)
    total = np.zeros(3, np.int32)
    for step, news in enumerate([[30, 7, 1], [8, 5, 20], [1, 12, 3], [16, 16, 16]]):
        cu, T, most = offsets(news), sum(news), max(news)
        parents = np.concatenate([np.arange(-1, n - 1) for n in news]) if step == 0 else random_trees(m.rng, news)
        lens = (total + np.array(news)).astype(np.int32)
        qkv, probs, uniform, tokens = m.inputs(T)
        before = [_host(m.cache, i) for i in range(LAYERS)]
        announce(f"drafted step {step} {half}")
        outs, kept, path, nxt = m.step(up(parents.astype(np.int32)), up(cu), up(lens), most, qkv, probs, uniform, tokens)
        words, pos = od.tree_ref(parents, cu, lens, -(-most // 32))
        want = od.verify_ref(host(probs), host(tokens), host(uniform), cu, most, parents)
        assert all(np.array_equal(host(a), b) for a, b in zip((kept, path, nxt), want))
        table, appended = host(m.table), []
        for i in range(LAYERS):
            x = qkv[i].float().cpu().numpy()
            w = [t.float().cpu().numpy() for t in m.w]
            k = od.rotate_ref(x[:, HQ:HQ + HKV], pos, m.angles, w[1])
            cache = o8.kv8_append_ref(k, x[:, HQ + HKV:], *before[i], table, cu, lens)
            q = o8.round_half(od.rotate_ref(x[:, :HQ], pos, m.angles, w[0]), half)
            o64, bound = o8.kv8_attention_rows(q, *cache, table, cu, lens, D ** -0.5, half, tree=words)
            assert np.all(np.abs(host(outs[i].float()) - o64) <= bound)
            appended.append(cache)
        clean = od.keep_ref(*(np.stack(c) for c in zip(*appended)), table, cu, lens, want[1], want[0])
        for i in range(LAYERS):
            assert all(np.array_equal(a, b[i]) for a, b in zip(_host(m.cache, i), clean))
        total = lens - np.array(news) + want[0]


def test_kept_drafts_are_as_good_as_appended_ones():
    """After a tree the cache holds what appending the kept tokens alone would have
    written, but for codes rounded to another page's scale: one step of a code."""
    a, b = Server(2, 1, 8), Server(2, 1, 8)
    n = 24
    parents = random_trees(a.rng, [n])
    qkv, probs, uniform, tokens = a.inputs(n)
    cu, lens = up(offsets([n])), up(np.array([n], np.int32))
    announce("kept drafts")
    probs.zero_()
    at = int(np.argmax(od.tree_ref(parents, offsets([n]), [n], 1)[1]))
    while at > 0:  # greedy rows along the deepest node's path
        probs[int(parents[at]), at] = 1
        at = int(parents[at])
    tokens.copy_(up(np.arange(n, dtype=np.int32)))
    _, kept, path, _ = a.step(up(parents), cu, lens, n, qkv, probs, uniform, tokens)
    m = int(kept[0])
    way = path[0, :m].long()
    assert m > 2
    sub = [x[way] for x in qkv]
    for i in range(LAYERS):
        q, k, v = sub[i].split([HQ, HKV, HKV], 1)
        mq.kv8_rope_append(q, k, v, *[t[i] for t in b.cache], b.table, up(offsets([m])), up(np.array([m], np.int32)), m,
                           b.cos_sin, q_weight=b.w[0], k_weight=b.w[1])
    for i in range(LAYERS):
        (ka, va, ksa, vsa), (kb, vb, ksb, vsb) = _host(a.cache, i), _host(b.cache, i)
        for t in range(m):
            p, r = int(a.table[0, t // PAGE]), t % PAGE
            for x, s, y, u in ((ka[p, :, r], ksa[p], kb[p, :, r], ksb[p]), (va[p, :, :, r], vsa[p], vb[p, :, :, r], vsb[p])):
                x, y = o8.e4m3_decode(x) * s[:, None], o8.e4m3_decode(y) * u[:, None]
                # each rounded once or twice: 2^-4 of the value, or half the smallest step of the larger scale
                step = np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10 * np.maximum(s, u)[:, None])
                assert np.all(np.abs(x - y) <= 3 * step)


def test_steps_captured():
    """One captured step, replayed while trees, lengths and inputs change and eager
    work runs between: every replay equals the eager step on a second server."""
    import torch
    seqs, n = 3, 9
    a, b = Server(3, seqs, 20), Server(3, seqs, 20)
    T = seqs * n
    cu = up(offsets([n] * seqs))
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    parents = up(random_trees(a.rng, [n] * seqs))
    qkv, probs, uniform, tokens = a.inputs(T)
    buf = a.buffers(T, n)
    announce("drafted step captured")
    warm = tuple(t.clone() for t in a.cache)
    a.step(parents, cu, lens, n, qkv, probs, uniform, tokens, buf)
    for t, w in zip(a.cache, warm):
        t.view(torch.uint8).copy_(w.view(torch.uint8))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(parents, cu, lens, n, qkv, probs, uniform, tokens, buf)
    for r in range(5):
        parents.copy_(up(random_trees(a.rng, [n] * seqs)))
        new = a.inputs(T)
        for x, y in zip(qkv, new[0]):
            x.copy_(y)
        for x, y in zip((probs, uniform, tokens), new[1:]):
            x.copy_(y)
        outs, kept, path, nxt = b.step(parents, cu, lens, n, qkv, probs, uniform, tokens)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(buf[f"o{i}"], outs[i]) for i in range(LAYERS)), f"replay {r}"
        assert torch.equal(buf["kept"], kept) and torch.equal(buf["path"], path) and torch.equal(buf["next"], nxt)
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a.cache, b.cache)), f"replay {r}"
        lens.copy_(lens + kept)


def test_steps_on_two_streams():
    import torch
    seqs, n = 2, 12
    cu = up(offsets([n] * seqs))
    one, two = [Server(s, seqs, 8) for s in (4, 5)], [Server(s, seqs, 8) for s in (4, 5)]
    work = [[(up(random_trees(m.rng, [n] * seqs)), m.inputs(seqs * n)) for _ in range(4)] for m in one]
    lens = [torch.full((seqs,), n + 5 * t, dtype=torch.int32, device="cuda") for t in range(4)]
    announce("drafted steps on two streams")
    want = [[m.step(p, cu, lens[t], n, *x)[:2] for t, (p, x) in enumerate(work[i])] for i, m in enumerate(one)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for t in range(4):
        for i, m in enumerate(two):
            p, x = work[i][t]
            with torch.cuda.stream(sides[i]):
                got[i].append(m.step(p, cu, lens[t], n, *x)[:2])
    torch.cuda.synchronize()
    for i in range(2):
        for (oa, ka), (ob, kb) in zip(got[i], want[i]):
            assert all(torch.equal(x, y) for x, y in zip(oa, ob)) and torch.equal(ka, kb)
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(one[i].cache, two[i].cache))


def test_stream_argument():
    """Every operator on a stream given to it: the results of the current one."""
    import torch
    a, b = Server(6, 1, 6), Server(6, 1, 6)
    n = 6
    cu, lens = up(offsets([n])), up(np.array([n], np.int32))
    parents = up(random_trees(a.rng, [n]))
    qkv, probs, uniform, tokens = a.inputs(n)
    want = a.step(parents, cu, lens, n, qkv, probs, uniform, tokens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    announce("drafted step, stream given")
    tree, pos = mq.kv8_tree_mask(parents, cu, lens, n, stream=s)
    for i in range(LAYERS):
        q, k, v = qkv[i].split([HQ, HKV, HKV], 1)
        layer = [t[i] for t in b.cache]
        q = mq.kv8_rope_append(q, k, v, *layer, b.table, cu, lens, n, b.cos_sin, positions=pos, q_weight=b.w[0],
                               k_weight=b.w[1], stream=s)
        o = mq.kv8_tree_attention(q, tree, *layer, b.table, cu, lens, n, stream=s)
        s.synchronize()
        assert torch.equal(o, want[0][i])
    kept, path, nxt = mq.draft_verify(probs, tokens, uniform, cu, n, parents=parents, stream=s)
    mq.kv8_tree_keep(*b.cache, b.table, cu, lens, path, kept, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((kept, path, nxt), want[1:]))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.cache, b.cache))
