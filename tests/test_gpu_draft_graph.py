"""Drafted tokens' operators captured in the forms that a small step does not take:
verification in two launches, trees of hundreds of nodes, prompts rotated in place,
several layers kept. Every replay, over other inputs and lengths, gives the bits of
an eager call."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from tests.draft_util import layered, offsets, random_trees, table_of_angles
from tests.fp8_util import codes_tensor, half_tensor
from tests.gpu_util import announce
from tests.kv8_util import up

pytestmark = pytest.mark.gpu


def _replays(call, state, enter, results, times=4):
    """`enter(i)` fills `state`'s tensors; `call` writes into some of them and returns
    others; compared are those that `results` picks from both."""
    import torch
    enter(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = call()
    for i in range(times):
        enter(i)
        saved = [t.clone() for t in state]
        eager = [t.clone() for t in results(call())]
        for t, s in zip(state, saved):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        got = results(captured)
        assert all(torch.equal(a, b) for a, b in zip(eager, got)), i


@pytest.mark.parametrize("draft", [False, True])
def test_verification_in_two_launches(draft):
    import torch
    rng = np.random.default_rng(1)
    B, n, V = 5, 6, 40001
    T = B * n
    assert mq.draft_verify_workspace_bytes(B, V, n) > 0
    g = torch.Generator(device="cuda").manual_seed(2)
    f32 = dict(dtype=torch.float32, device="cuda")
    probs, q, uniform = torch.zeros((T, V), **f32), torch.zeros((T, V), **f32), torch.zeros(T, **f32)
    tokens, parents, cu = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (T, T, B + 1))

    def enter(i):
        probs.copy_(torch.softmax(4 * torch.randn((T, V), generator=g, device="cuda"), -1))
        q.copy_(torch.softmax(probs.log() + 0.5 * torch.randn((T, V), generator=g, device="cuda"), -1))
        uniform.copy_(torch.rand(T, generator=g, device="cuda"))
        news = [n] * B if i == 0 else [int(x) for x in rng.integers(0, n + 1, B)]
        cu.copy_(up(offsets(news)))
        parents[:sum(news)] = up(random_trees(rng, news))
        tokens.copy_((q if draft else probs).argmax(-1).int().roll(1))

    announce(f"draft_verify captured, V={V}, draft={draft}")
    _replays(lambda: mq.draft_verify(probs, tokens, uniform, cu, n, **({"draft_probs": q} if draft else {"parents": parents})),
             [probs, q, uniform, tokens, parents, cu], enter, lambda r: r)


def test_masks_of_large_trees():
    import torch
    rng = np.random.default_rng(2)
    B, most = 7, 600
    T = B * most
    i32 = dict(dtype=torch.int32, device="cuda")
    parents, cu, lens = torch.zeros(T, **i32), torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    mask, pos = torch.zeros((T, 19), **i32), torch.zeros(T, **i32)

    def enter(i):
        news = [int(x) for x in rng.integers(0, most + 1, B)]
        parents[:sum(news)] = up(random_trees(rng, news, back=40))
        cu.copy_(up(offsets(news)))
        lens.copy_(up(np.array(news, np.int32) + 9))
        mask.fill_(7)
        pos.fill_(7)

    announce("kv8_tree_mask captured")
    _replays(lambda: mq.kv8_tree_mask(parents, cu, lens, most, mask=mask, positions=pos), [parents, cu, lens, mask, pos], enter,
             lambda r: r)


@pytest.mark.parametrize("D,page", [(64, 64), (128, 16)])
def test_prompts_in_place_then_kept(D, page):
    """k and v of two layers' caches appended from one tensor whose q turns in place, then a path kept."""
    import torch
    rng = np.random.default_rng(D)
    B, most, Hq, H, layers = 3, 200, 6, 2, 2
    T, longest = B * most, 500
    cache, table = layered(rng, layers, [longest] * B, H, page, D)
    dev = [codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])]
    first = [t.view(torch.uint8).clone() for t in dev]
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, lens, kept, path = torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros((B, most), **i32)
    qkv = half_tensor(np.zeros((layers, T, Hq + 2 * H, D)), "bf16")[0]
    angles, where = up(table_of_angles(rng, longest, D)), up(table)
    w = [half_tensor(rng.uniform(0.5, 1.5, D), "bf16")[0] for _ in "qk"]

    def enter(i):
        news = [int(x) for x in rng.integers(1, most + 1, B)]
        cu.copy_(up(offsets(news)))
        lens.copy_(up(np.array([n + int(rng.integers(0, longest - most)) for n in news], np.int32)))
        m = [int(rng.integers(1, n + 1)) for n in news]
        way = np.full((B, most), -1, np.int32)
        for b in range(B):
            way[b, :m[b]] = [0] + sorted(1 + rng.choice(news[b] - 1, m[b] - 1, replace=False)) if m[b] > 1 else [0]
        path.copy_(up(way))
        kept.copy_(up(np.array(m, np.int32)))
        qkv.copy_(half_tensor(rng.standard_normal(tuple(qkv.shape)), "bf16")[0])
        for t, s in zip(dev, first):
            t.view(torch.uint8).copy_(s)

    def call():
        for i in range(layers):
            q, k, v = qkv[i].split([Hq, H, H], 1)
            mq.kv8_rope_append(q, k, v, *[t[i] for t in dev], where, cu, lens, most, angles, q_weight=w[0], k_weight=w[1], out=q)
        mq.kv8_tree_keep(*dev, where, cu, lens, path, kept)

    state = [t.view(torch.uint8) for t in dev] + [cu, lens, kept, path, qkv.view(torch.int16)]
    announce(f"kv8_rope_append in place and kv8_tree_keep captured, D={D}")
    _replays(call, state, enter, lambda _: state)
