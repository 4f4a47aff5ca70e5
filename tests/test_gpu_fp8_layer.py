"""The 8-bit operators as a model runs them, an attention block: RMS norm with
the residual to e4m3 codes, the fused qkv product, append to the paged cache,
attention over it, the output projection. Every stage of a ragged prompt and of
the decode steps after it is checked against its oracle on the inputs it got;
captured decode steps and blocks on two streams at once give the eager bits."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import codes_of, codes_tensor, group_max_sum, half_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu

EPS = 1e-5
HQ, HKV, D, PAGE, HIDDEN = 8, 2, 128, 16, 1024
QKV = (HQ + 2 * HKV) * D


def _up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Block:
    """Weights and cache of one attention block."""

    def __init__(self, seed, half, seqs, pages):
        import torch
        rng = np.random.default_rng(seed)
        self.half, self.rng = half, rng
        self.dt = torch.bfloat16 if half == "bf16" else torch.float16

        def weight(n, k):
            w = rng.standard_normal((n, k)) * k ** -0.5
            s = np.full((-(-n // 128), -(-k // 128)), 4 * k ** -0.5 / 448, np.float32)
            q = o8.e4m3_encode(np.clip(w / s[0, 0], -448, 448))
            return q, s

        self.wqkv, self.wo = weight(QKV, HIDDEN), weight(HIDDEN, HQ * D)
        self.t = {n: (codes_tensor(q), _up(s)) for n, (q, s) in (("qkv", self.wqkv), ("o", self.wo))}
        self.norm, self.normf = half_tensor(1 + 0.1 * rng.standard_normal(HIDDEN), half)
        P = seqs * pages + 2
        self.table = _up(rng.permutation(P)[:seqs * pages].reshape(seqs, pages).astype(np.int32))
        self.cache = (torch.zeros((P, HKV, PAGE, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                      torch.zeros((P, HKV, D, PAGE), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                      torch.zeros((P, HKV), device="cuda"), torch.zeros((P, HKV), device="cuda"))

    def input(self, T):
        return [half_tensor(self.rng.standard_normal((T, HIDDEN)) * a, self.half)[0] for a in (1.0, 2.0)]

    def run(self, x, residual, cu, lens, max_q, buffers=None, see=None):
        """One block; `buffers`: caller-owned outputs and workspaces."""
        b = buffers or {}
        seen = see or (lambda *a: None)
        T = x.shape[0]
        xq, s_x, h = mq.rmsnorm_fp8(x, self.norm, EPS, residual, out=b.get("xq"), s_out=b.get("s_x"), h_out=b.get("h"))
        qkv = mq.fp8_block_mm(xq, s_x, *self.t["qkv"], out=b.get("qkv"), workspace=b.get("w1"), out_dtype=self.dt)
        q = qkv[:, :HQ * D].view(T, HQ, D)
        k = qkv[:, HQ * D:(HQ + HKV) * D].view(T, HKV, D)
        v = qkv[:, (HQ + HKV) * D:].view(T, HKV, D)
        seen("norm", x, residual, xq, s_x, h)
        seen("qkv", xq, s_x, qkv)
        seen("before", k, v)
        mq.kv8_append(k, v, *self.cache, self.table, cu, lens, max_q_len=max_q)
        seen("append", k, v)
        o = mq.kv8_attention(q, *self.cache, self.table, cu, lens, max_q_len=max_q, out=b.get("o"), workspace=b.get("w2"))
        seen("attention", q, o)
        y = mq.fp8_linear(o.view(T, HQ * D), *self.t["o"], out=b.get("y"), workspace=b.get("w3"))
        seen("o", o, y)
        return y, h

    def buffers(self, T, seqs, max_q):
        import torch
        u8 = dict(dtype=torch.uint8, device="cuda")
        half = dict(dtype=self.dt, device="cuda")
        kb = HIDDEN // 128
        return {"xq": torch.empty((T, HIDDEN), **u8).view(torch.float8_e4m3fn), "s_x": torch.empty((kb, T), device="cuda"),
                "h": torch.empty((T, HIDDEN), **half), "qkv": torch.empty((T, QKV), **half),
                "o": torch.empty((T, HQ, D), **half), "y": torch.empty((T, HIDDEN), **half),
                "w1": torch.empty(mq.fp8_block_mm_workspace_bytes(T, QKV, HIDDEN) + 16, **u8),
                "w2": torch.empty(mq.kv8_attention_workspace_bytes(T, seqs, HQ, HKV, D, PAGE, self.table.shape[1], max_q) + 16,
                                  **u8),
                "w3": torch.empty(mq.fp8_linear_workspace_bytes(T, HIDDEN, HQ * D) + 16, **u8)}


def _host_cache(cache):
    return codes_of(cache[0]), codes_of(cache[1]), host(cache[2]), host(cache[3])


def _mm_ok(xq, s_x, w, y, half, what):
    y64, mag = o8.fp8_mm_ref(xq, s_x, *w)
    bound = o8.fp8_mm_bound(y64, mag, group_max_sum(xq, s_x, *w), xq.shape[1], half)
    over = np.abs(host(y.float()) - y64) / bound
    assert np.all(over <= 1.0), f"{what}: worst err/bound {over.max():.3g}"


@pytest.mark.parametrize("half", ["fp16", "bf16"])
def test_block_stages(half):
    """A ragged prompt (one sequence joins later), then decode steps of all."""
    seqs = 3
    m = Block(1, half, seqs, 12)
    before = {}

    def see(cu, lens):
        def f(stage, *a):
            announce(f"block {half} {stage}")
            if stage == "norm":
                x, residual, xq, s_x, h = a
                v, hh = o8.rmsnorm_ref(host(x.float()), m.normf, EPS, host(residual.float()), half)
                codes, s = o8.quant_fp8_blocks_ref(v)
                assert np.array_equal(codes_of(xq), codes) and np.array_equal(host(s_x), s)
                assert np.array_equal(host(h.float()), hh)
            elif stage == "qkv":
                _mm_ok(codes_of(a[0]), host(a[1]), m.wqkv, a[2], half, "qkv")
            elif stage == "before":
                before["cache"] = _host_cache(m.cache)
            elif stage == "append":
                want = o8.kv8_append_ref(host(a[0].float()), host(a[1].float()), *before["cache"], host(m.table), cu, lens)
                got = _host_cache(m.cache)
                assert all(np.array_equal(g, w) for g, w in zip(got, want))
            elif stage == "attention":
                cache = _host_cache(m.cache)
                q = host(a[0].float())
                o64, mag, sub = o8.kv8_attention_ref(q, *cache, host(m.table), cu, lens, D ** -0.5)
                bound = o8.kv8_attention_bound(q, 448.0 * float(cache[2].max()), D ** -0.5, D, max(lens), o64, mag, sub, half)
                assert np.all(np.abs(host(a[1].float()) - o64) <= bound)
            else:
                o, y = a
                codes, s = o8.quant_fp8_blocks_ref(host(o.float()).reshape(len(o), -1))
                _mm_ok(codes, s, m.wo, y, half, "o")
        return f

    lens = np.zeros(seqs, np.int32)
    for step, news in enumerate([[90, 33, 0], [1, 1, 70], [1, 1, 1], [1, 1, 1], [16, 2, 1]]):
        cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        lens = (lens + np.array(news)).astype(np.int32)
        x, residual = m.input(int(cu[-1]))
        m.run(x, residual, _up(cu), _up(lens), max(news), see=see(cu, lens))


@pytest.mark.parametrize("seqs,new", [(3, 1), (2, 40)])
def test_block_captured(seqs, new):
    """One captured step, replayed while lengths, tables and inputs change and
    eager steps run between: every replay equals the eager step on a second
    cache, bit for bit."""
    import torch
    a, b = Block(2, "bf16", seqs, 40), Block(2, "bf16", seqs, 40)
    T = seqs * new
    cu = _up((np.arange(seqs + 1) * new).astype(np.int32))
    lens = torch.full((seqs,), new, dtype=torch.int32, device="cuda")
    x, residual = a.input(T)
    buf = a.buffers(T, seqs, new)
    announce(f"block captured, {seqs} x {new}")
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
        for t, u in zip((x, residual), a.input(T)):
            t.copy_(u)
        y, h = b.run(x, residual, cu, lens, new)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf["y"], y) and torch.equal(buf["h"], h), f"replay {r}"
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a.cache, b.cache)), f"replay {r}"


def test_blocks_on_two_streams():
    """Two blocks on two streams at once: the bits of one after the other."""
    import torch
    seqs, steps = 4, 6
    one = [Block(s, "fp16", seqs, 20) for s in (3, 4)]
    two = [Block(s, "fp16", seqs, 20) for s in (3, 4)]
    cu = _up(np.arange(seqs + 1, dtype=np.int32))
    xs = [[m.input(seqs) for _ in range(steps)] for m in one]
    lens = [torch.full((seqs,), 1 + t, dtype=torch.int32, device="cuda") for t in range(steps)]
    announce("blocks on two streams")
    want = [[m.run(*xs[i][t], cu, lens[t], 1)[0] for t in range(steps)] for i, m in enumerate(one)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for t in range(steps):
        for i, m in enumerate(two):
            with torch.cuda.stream(sides[i]):
                got[i].append(m.run(*xs[i][t], cu, lens[t], 1)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
