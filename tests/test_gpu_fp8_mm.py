"""The e4m3 product with a scale per block of 128 on an MI355X against the
float64 oracle, within the bound derived for its arithmetic
(``oracle.fp8.fp8_mm_bound``): every kernel form's edges, ragged M, N and K,
one-hot rows (exact), scales over a wide range, graph replay, another stream,
and the layer fp8_linear bit for bit its two parts."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import activations, codes_of, codes_tensor, group_max_sum, half_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu


def _dt(half):
    import torch
    return torch.bfloat16 if half == "bf16" else torch.float16


def _up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _inputs(rng, M, N, K, wide=False):
    xq = o8.e4m3_encode(np.clip(rng.standard_normal((M, K)) * 100, -448, 448))
    wq = o8.e4m3_encode(np.clip(rng.standard_normal((N, K)) * 100, -448, 448))
    kb, nb = -(-K // 128), -(-N // 128)
    if wide:
        sx, sw = np.exp2(rng.uniform(-14, 2, (kb, M))), np.exp2(rng.uniform(-18, -4, (nb, kb)))
    else:
        sx, sw = rng.uniform(2e-3, 8e-3, (kb, M)), rng.uniform(1e-4, 4e-4, (nb, kb))
    return xq, sx.astype(np.float32), wq, sw.astype(np.float32)


def _check(xq, sx, wq, sw, half, what, rows=None):
    M, K = xq.shape
    announce(f"fp8_block_mm {what} {half} M={M} N={wq.shape[0]} K={K}")
    y = mq.fp8_block_mm(codes_tensor(xq), _up(sx), codes_tensor(wq), _up(sw), out_dtype=_dt(half))
    y = host(y.float()).astype(np.float64)
    if rows is not None:
        y, xq, sx = y[rows], xq[rows], sx[:, rows]
    y64, mag = o8.fp8_mm_ref(xq, sx, wq, sw)
    gmax = group_max_sum(xq, sx, wq, sw)
    over = np.abs(y - y64) / o8.fp8_mm_bound(y64, mag, gmax, K, half)
    assert np.all(over <= 1.0), f"{what}: worst err/bound {over.max():.3g} at {np.unravel_index(over.argmax(), over.shape)}"
    return y


# one token to past the largest decode form, then the tiled forms
SHAPES = [(1, 16, 16), (1, 1, 128), (2, 9000, 512), (11, 700, 12288), (16, 8200, 4096), (16, 100, 12288), (20, 17, 16), (1, 4096, 4096), (3, 130, 144), (5, 300, 1040), (15, 257, 2064), (16, 512, 4096),
          (17, 384, 1152), (32, 129, 2048), (33, 640, 4096), (63, 1000, 784), (64, 256, 12288), (65, 131, 272),
          (100, 1024, 1024), (255, 300, 144), (256, 4096, 512), (300, 9000, 640), (517, 6144, 1040),
          (1030, 3000, 400), (1500, 13000, 272), (4100, 4100, 160)]


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mm_bound(M, N, K, half):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    _check(*_inputs(rng, M, N, K), half, "random")


@pytest.mark.parametrize("M,N,K", [(4, 300, 1552), (40, 200, 1552), (200, 300, 1552), (900, 16400, 272)])
def test_mm_wide_scales(M, N, K):
    rng = np.random.default_rng(M + N)
    _check(*_inputs(rng, M, N, K, wide=True), "bf16", "wide scales")


@pytest.mark.parametrize("M,N,K", [(2, 200, 1040), (33, 200, 1040), (130, 260, 1040), (700, 20000, 272)])
def test_mm_one_hot_is_exact(M, N, K):
    """Row m of xq holds one 1.0 at k = k(m): y picks weight k of every
    channel, rounded once; a wrong block, scale or layout shows at once."""
    rng = np.random.default_rng(M)
    _, sx, wq, sw = _inputs(rng, M, N, K)
    ks = rng.integers(0, K, M)
    xq = np.zeros((M, K), np.uint8)
    xq[np.arange(M), ks] = o8.e4m3_encode([1.0])[0]
    announce(f"fp8_block_mm one-hot M={M} N={N} K={K}")
    y = host(mq.fp8_block_mm(codes_tensor(xq), _up(sx), codes_tensor(wq), _up(sw), out_dtype=_dt("bf16")).float())
    sc = sx[ks // 128, np.arange(M)][:, None] * sw[np.arange(N) // 128][:, ks // 128].T  # fl32
    want = o8.round_half((o8.e4m3_decode(wq[:, ks]).T.astype(np.float32) * sc).astype(np.float32), "bf16")
    assert np.array_equal(y, want)


def test_mm_every_code():
    """Every pair of finite codes meets in some product: K = 254 products of
    x's code i with w's code (i + n) mod 254, summed against the oracle."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    xq = np.zeros((3, 256), np.uint8)
    xq[:, :254] = codes
    wq = np.zeros((254, 256), np.uint8)
    for n in range(254):
        wq[n, :254] = np.roll(codes, n)
    one = np.ones((2, 3), np.float32), np.full((2, 2), 2.0 ** -6, np.float32)
    _check(xq, one[0], wq, one[1], "fp16", "every code (decode form)")
    xq = np.repeat(xq[:1], 80, 0)
    _check(xq, np.ones((2, 80), np.float32), wq, one[1], "fp16", "every code (tiled form)")


def test_mm_rows_do_not_mix():
    """A row's result does not depend on the rows beside it (same form)."""
    import torch
    rng = np.random.default_rng(12)
    xq, sx, wq, sw = _inputs(rng, 300, 400, 656)
    a = mq.fp8_block_mm(codes_tensor(xq), _up(sx), codes_tensor(wq), _up(sw))
    perm = rng.permutation(300)
    b = mq.fp8_block_mm(codes_tensor(xq[perm]), _up(sx[:, perm]), codes_tensor(wq), _up(sw))
    assert torch.equal(a[torch.from_numpy(perm).cuda()], b)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 520, 1040), (48, 1024, 4096), (333, 700, 2064)])
def test_linear_is_its_parts(M, N, K, half):
    import torch
    rng = np.random.default_rng(M + N + K)
    t, x = half_tensor(activations(rng, M, K), half)
    _, _, wq, sw = _inputs(rng, 1, N, K)
    wt, st = codes_tensor(wq), _up(sw)
    announce(f"fp8_linear {half} M={M} N={N} K={K}")
    y = mq.fp8_linear(t, wt, st)
    q, s = mq.quant_fp8_blocks(t)
    assert torch.equal(y, mq.fp8_block_mm(q, s, wt, st, out_dtype=_dt(half)))
    y64, mag = o8.fp8_mm_ref(codes_of(q), host(s), wq, sw)
    gmax = group_max_sum(codes_of(q), host(s), wq, sw)
    assert np.all(np.abs(host(y.float()) - y64) <= o8.fp8_mm_bound(y64, mag, gmax, K, half))


def test_empty():
    import torch
    e = codes_tensor(np.zeros((0, 256), np.uint8))
    w, sw = codes_tensor(np.zeros((128, 256), np.uint8)), torch.zeros((1, 2), device="cuda")
    assert mq.fp8_block_mm(e, torch.zeros((2, 0), device="cuda"), w, sw).shape == (0, 128)
    assert mq.fp8_linear(torch.zeros((0, 256), dtype=torch.float16, device="cuda"), w, sw).shape == (0, 128)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_graph_replays_and_stream(M):
    import torch
    rng = np.random.default_rng(M)
    K, N = 2064, 900
    t, _ = half_tensor(activations(rng, M, K), "bf16")
    _, _, wq, sw = _inputs(rng, 1, N, K)
    wt, st = codes_tensor(wq), _up(sw)
    ws = torch.empty(max(mq.fp8_linear_workspace_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda")
    y = mq.fp8_linear(t, wt, st, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.fp8_linear(t, wt, st, out=y, workspace=ws)
    side = torch.cuda.Stream()
    for _ in range(3):
        t.copy_(half_tensor(activations(rng, M, K), "bf16")[0])
        want = mq.fp8_linear(t, wt, st)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        side.wait_stream(torch.cuda.current_stream())
        other = mq.fp8_linear(t, wt, st, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, want)
