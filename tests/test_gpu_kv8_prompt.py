"""The prompt form of attention where other tests of the same calls take the
form of few rows: outputs that are not split, caches past 4 GB, captured calls
whose lengths change. Every call says which form it takes."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import codes_tensor, half_tensor
from tests.gpu_util import announce
from tests.kv8_util import check_rows, empty_cache, up
from tests.test_gpu_fp8_layer import D as BLOCK_D, HKV, HQ, PAGE, Block

pytestmark = pytest.mark.gpu


def _random_codes(rng, shape):
    return o8.e4m3_encode(np.clip(rng.standard_normal(shape) * 90, -448, 448))


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 64)])
def test_unsplit(page, D, half):
    """256 row tiles: no splits. Ragged sequences of up to 40 new tokens, some
    without any, over up to 700 keys."""
    rng = np.random.default_rng(page + D)
    B, Hkv, G, most, width = 32, 4, 8, 40, -(-720 // page)
    news = [most, 1, 0, 33] + [int(n) for n in rng.integers(30, most + 1, B - 4)]
    totals = [700, 64, 5, 33] + [n + int(t) for n, t in zip(news[4:], rng.integers(0, 130, B - 4))]
    T = B * most  # (rows behind the last sequence)
    assert mq.kv8_attention_form(T, B, G * Hkv, Hkv, D, page, width, most) == "prompt"
    assert mq.kv8_attention_workspace_bytes(T, B, G * Hkv, Hkv, D, page, width, most) == 0
    need = [-(-t // page) for t in totals]
    P = sum(need)
    cache = empty_cache(P, Hkv, page, D)
    cache[0][:], cache[1][:] = _random_codes(rng, cache[0].shape), _random_codes(rng, cache[1].shape)
    cache[2][:], cache[3][:] = (np.exp2(rng.integers(-9, -5, (P, Hkv))) for _ in range(2))
    table = np.full((B, width), -1, np.int32)
    ids = rng.permutation(P)
    for b, n in enumerate(need):
        table[b, :n], ids = ids[:n], ids[n:]
    cu = np.concatenate([[0], np.cumsum(news)])
    check_rows(rng.standard_normal((T, G * Hkv, D)), half, cache, table, cu, totals, "unsplit",
               fro=1e-3 if half == "fp16" else 5e-3)


@pytest.mark.parametrize("new,total,width", [(100, 150, 4096), (1100, 1100, 18)])
def test_cache_past_four_gigabytes(new, total, width):
    """Pages whose byte offsets pass 2^32: the bits of the same pages in a small
    pool. Split and unsplit."""
    import torch
    H, G, D, page, P = 8, 4, 128, 64, 70000  # 4.6 GB of K codes, as many of V
    assert mq.kv8_attention_form(new, 1, G * H, H, D, page, width, new) == "prompt"
    assert (mq.kv8_attention_workspace_bytes(new, 1, G * H, H, D, page, width, new) > 0) == (new == 100)
    rng = np.random.default_rng(new)
    n = -(-total // page)
    ids = np.array([P - 1 - 3 * i if i != 1 else 2 for i in range(n)])
    kc = torch.empty((P, H, page, D), dtype=torch.uint8, device="cuda")
    vc = torch.empty((P, H, D, page), dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones((P, H), device="cuda"), torch.ones((P, H), device="cuda")
    at = torch.from_numpy(ids).cuda()
    small = (up(_random_codes(rng, (n, H, page, D))), up(_random_codes(rng, (n, H, D, page))),
             up(np.exp2(rng.integers(-9, -5, (n, H))).astype(np.float32)),
             up(np.exp2(rng.integers(-9, -5, (n, H))).astype(np.float32)))
    for far, near in zip((kc, vc, ks, vs), small):
        far[at] = near
    tables = np.full((2, 1, width), -1, np.int32)
    tables[0, 0, :n], tables[1, 0, :n] = ids, range(n)
    q, _ = half_tensor(rng.standard_normal((new, G * H, D)), "bf16")
    args = up(np.array([0, new], np.int32)), up(np.array([total], np.int32))
    e4m3 = torch.float8_e4m3fn
    announce(f"kv8 past 4 GB: prompt of {new}")
    got = mq.kv8_attention(q, kc.view(e4m3), vc.view(e4m3), ks, vs, up(tables[0]), *args, max_q_len=new)
    want = mq.kv8_attention(q, small[0].view(e4m3), small[1].view(e4m3), *small[2:], up(tables[1]), *args, max_q_len=new)
    assert torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("B,new,H,G,D,page,width", [(3, 40, 2, 4, 128, 16, 4096), (4, 512, 8, 8, 64, 64, 40)])
def test_graph_replays_with_changing_lengths(B, new, H, G, D, page, width):
    """Append and attention captured once; between replays lengths, tables and
    inputs change, with eager calls in between. Split and unsplit."""
    import torch
    rng = np.random.default_rng(new)
    T, used = B * new, 40
    P = B * used + 3
    assert mq.kv8_attention_form(T, B, G * H, H, D, page, width, new) == "prompt"
    need = mq.kv8_attention_workspace_bytes(T, B, G * H, H, D, page, width, new)
    assert (need > 0) == (new == 40)
    a = tuple(codes_tensor(c) if c.dtype == np.uint8 else up(c) for c in empty_cache(P, H, page, D))
    b = tuple(t.clone() for t in a)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    cu = up((np.arange(B + 1) * new).astype(np.int32))
    lens = torch.full((B,), new, dtype=torch.int32, device="cuda")
    q, _ = half_tensor(rng.standard_normal((T, H * G, D)), "bf16")
    kv, _ = half_tensor(rng.standard_normal((T, 2, H, D)), "bf16")
    out = torch.empty_like(q)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step(cache, o, w):
        mq.kv8_append(kv[:, 0], kv[:, 1], *cache, table, cu, lens, max_q_len=new)
        mq.kv8_attention(q, *cache, table, cu, lens, max_q_len=new, out=o, workspace=w)

    table[:, :used] = up(rng.permutation(P)[:B * used].reshape(B, used).astype(np.int32))
    announce(f"kv8 graph, prompts of {new}")
    step(tuple(t.clone() for t in a), out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, out, ws)
    for r in range(4):
        if r == 2:  # the sequences start over in other pages
            table[:, :used] = up(rng.permutation(P)[:B * used].reshape(B, used).astype(np.int32))
        lens.copy_(torch.tensor([new * (1 + r % 2), new, new + 9 * (r % 2)] + [new] * (B - 3), dtype=torch.int32))
        q.copy_(half_tensor(rng.standard_normal((T, H * G, D)), "bf16")[0])
        kv.copy_(half_tensor(rng.standard_normal((T, 2, H, D)) * (1 + 3 * r), "bf16")[0])
        eager = torch.empty_like(out)
        step(b, eager, None)
        g.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(eager).all() and torch.equal(out, eager), f"replay {r}"
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b)), f"replay {r}: cache"


def test_block_captured():
    """The whole attention block captured with prompts of 40 tokens under wide
    tables, replayed while lengths and inputs change."""
    import torch
    seqs, new, width = 2, 40, 4096
    assert mq.kv8_attention_form(seqs * new, seqs, HQ, HKV, BLOCK_D, PAGE, width, new) == "prompt"
    a, b = Block(2, "bf16", seqs, width), Block(2, "bf16", seqs, width)
    cu = up((np.arange(seqs + 1) * new).astype(np.int32))
    lens = torch.full((seqs,), new, dtype=torch.int32, device="cuda")
    x, residual = a.input(seqs * new)
    buf = a.buffers(seqs * new, seqs, new)
    announce(f"block captured, prompts of {new}")
    warm = tuple(t.clone() for t in a.cache)
    a.run(x, residual, cu, lens, new, buf)
    for t, w in zip(a.cache, warm):
        t.view(torch.uint8).copy_(w.view(torch.uint8))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(x, residual, cu, lens, new, buf)
    for r in range(5):
        lens.copy_(torch.tensor([new * (r + 1) + 7 * r * (s == 0) for s in range(seqs)], dtype=torch.int32))
        for t, u in zip((x, residual), a.input(seqs * new)):
            t.copy_(u)
        y, h = b.run(x, residual, cu, lens, new)
        g.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(y).all() and torch.equal(buf["y"], y) and torch.equal(buf["h"], h), f"replay {r}"
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a.cache, b.cache)), f"replay {r}"
