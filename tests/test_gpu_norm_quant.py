"""RMS norm with 8-bit output and the e4m3 quantizer on an MI355X: codes,
scales and the residual sum bit-exact against the oracle, at every register
form's edges, short last blocks, ties, zero and tiny rows; in place, on another
stream, captured, and followed by the int8 and e4m3 products."""

import numpy as np
import pytest

import oracle
import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import activations, codes_of, half_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu

EPS = 1e-5
HALVES = ["fp16", "bf16"]


def _check_norm(x, w, res, half, fp8, what, eps=EPS):
    announce(f"rmsnorm {what} {half} fp8={fp8} residual={res is not None} shape={x.shape}")
    tx, x = half_tensor(x, half)
    tw, w = half_tensor(w, half)
    tr = None
    if res is not None:
        tr, res = half_tensor(res, half)
    got = (mq.rmsnorm_fp8 if fp8 else mq.rmsnorm_int8)(tx, tw, eps, residual=tr)
    v, h = o8.rmsnorm_ref(x, w, eps, res, half)
    q, s = o8.quant_fp8_blocks_ref(v) if fp8 else oracle.quant_per_token_int8_ref(v)
    gs = host(got[1])
    assert np.array_equal(gs.view(np.uint32), s.view(np.uint32)), f"{what}: scales differ"
    gq = codes_of(got[0]) if fp8 else host(got[0])
    bad = np.argwhere(gq != q)
    assert bad.size == 0, f"{what}: {len(bad)} codes differ, first at {bad[:3].tolist()}"
    if res is not None:
        assert np.array_equal(host(got[2].float()), h), f"{what}: h differs"
    else:
        assert len(got) == 2


# every register form's first and last K, short last blocks, odd row counts
SHAPES = [(1, 16), (5, 496), (4, 512), (6, 528), (3, 2048), (2, 2064), (130, 4096), (1, 4096), (3, 4112), (5, 8192),
          (2, 8208), (2, 16384), (2, 16400), (1, 32768), (2, 32784), (1, 65536), (333, 5008)]


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("half", HALVES)
@pytest.mark.parametrize("M,K", SHAPES)
def test_norm_bitexact(M, K, half, fp8, residual):
    rng = np.random.default_rng(M * 100003 + K)
    x = activations(rng, M, K)
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    _check_norm(x, w, 3 * rng.standard_normal((M, K)) if residual else None, half, fp8, "random")


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
@pytest.mark.parametrize("half", HALVES)
def test_norm_edge_rows(half, fp8):
    K = 272
    rng = np.random.default_rng(9)
    big, tiny = (60000.0, 6e-8) if half == "fp16" else (3e38, 1e-38)
    rows = [np.zeros(K), np.full(K, tiny), np.full(K, big), np.resize([1.0, -1.0], K), np.resize([big, tiny, 0.0, -tiny], K),
            np.concatenate([np.zeros(128), np.ones(K - 128)]), np.resize(np.arange(-8, 9), K) / 8.0,
            np.concatenate([[1.0], np.zeros(K - 1)])]
    x = np.array(rows, np.float32)
    w = np.resize([1.0, 0.5, -2.0, 0.0, 1.0], K).astype(np.float32)
    _check_norm(x, w, None, half, fp8, "edges")
    # the sum cancels to zero, and to the least bit of the larger
    res = -x.copy()
    res[3] = -x[3] + rng.standard_normal(K)
    _check_norm(x, w, res, half, fp8, "cancelling residual")


def test_norm_zero_row_without_eps():
    tx, _ = half_tensor(np.zeros((2, 64)), "fp16")
    tw, _ = half_tensor(np.ones(64), "fp16")
    for fn in (mq.rmsnorm_int8, mq.rmsnorm_fp8):
        q, s = fn(tx, tw, 0.0)
        assert not host(s).any() and not host(q.view(__import__("torch").int8)).any()


@pytest.mark.parametrize("half", HALVES)
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (65, 4096), (7, 12288), (1000, 272), (1, 131072 + 16)])
def test_quant_fp8_blocks_bitexact(M, K, half):
    rng = np.random.default_rng(M + K)
    t, x = half_tensor(activations(rng, M, K), half)
    announce(f"quant_fp8_blocks {half} {M}x{K}")
    q, s = mq.quant_fp8_blocks(t)
    rq, rs = o8.quant_fp8_blocks_ref(x)
    assert np.array_equal(host(s).view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes_of(q), rq)


@pytest.mark.parametrize("half", HALVES)
def test_quant_fp8_blocks_ties_and_extremes(half):
    """Quotients that sit on, and one binary32 step beside, the borders of
    e4m3 codes; subnormal codes; blocks of zeros, of the smallest and the
    largest values of the format."""
    rng = np.random.default_rng(5)
    rows = []
    mids = [(8 + m + 0.5) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8) if (8 + m + 0.5) / 8 * 2.0 ** e < 448]
    rows.append(np.resize(np.array([448.0] + mids), 256))
    rows.append(np.resize(np.array([448.0] + [(j + 0.5) * 2.0 ** -9 for j in range(8)]), 256))
    for a in (1.0, 1.25, 1.5, 3.0, 5.0):
        rows.append(np.resize(np.concatenate([[a], a * np.arange(1, 64) / 128]), 256))
    rows.append(np.zeros(256))
    tiny = 6e-8 if half == "fp16" else 1e-40
    rows.append(np.resize([tiny, -tiny, 0.0], 256))
    rows.append(np.resize([65504.0, -65504.0, 1.0] if half == "fp16" else [3.38e38, -3.38e38, 1e30], 256))
    rows.append(np.resize([-0.0, 0.0, 1.0], 256))
    t, x = half_tensor(np.array(rows) * np.where(rng.random((len(rows), 256)) < 0.5, 1.0, -1.0), half)
    announce(f"quant_fp8_blocks ties {half}")
    q, s = mq.quant_fp8_blocks(t)
    rq, rs = o8.quant_fp8_blocks_ref(x)
    assert np.array_equal(host(s).view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes_of(q), rq)


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
def test_norm_residual_in_place_and_stream(fp8):
    import torch
    rng = np.random.default_rng(6)
    tx, x = half_tensor(rng.standard_normal((40, 4096)), "bf16")
    tr, r = half_tensor(rng.standard_normal((40, 4096)), "bf16")
    tw, w = half_tensor(rng.standard_normal(4096), "bf16")
    fn = mq.rmsnorm_fp8 if fp8 else mq.rmsnorm_int8
    q0, s0, h0 = fn(tx, tw, EPS, residual=tr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q1, s1, h1 = fn(tx, tw, EPS, residual=tr, h_out=tr, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert h1 is tr and torch.equal(h0, tr) and torch.equal(s0, s1)
    assert torch.equal(q0.view(torch.uint8), q1.view(torch.uint8))


def test_norm_feeds_the_int8_product():
    """rmsnorm_int8 -> w8a8_scaled_mm, bit for bit the same as quantizing the
    oracle's normed rows."""
    import torch
    rng = np.random.default_rng(8)
    tx, x = half_tensor(activations(rng, 70, 1024), "fp16")
    tw, w = half_tensor(rng.uniform(0.5, 1.5, 1024), "fp16")
    wq, s_ch = oracle.quant_per_token_int8_ref((0.02 * rng.standard_normal((256, 1024))).astype(np.float16))
    q, s = mq.rmsnorm_int8(tx, tw, EPS)
    y = host(mq.w8a8_scaled_mm(q, s, torch.from_numpy(wq).cuda(), torch.from_numpy(s_ch).cuda()))
    v, _ = o8.rmsnorm_ref(x, w, EPS)
    want = oracle.w8a8_ref(*oracle.quant_per_token_int8_ref(v), wq, s_ch)
    assert np.all(np.abs(y.astype(np.float64) - want) <= 2.0 ** -11 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -20 * np.abs(want) + 2.0 ** -25)


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
def test_norm_graph_replays(fp8):
    import torch
    rng = np.random.default_rng(10)
    tx, _ = half_tensor(rng.standard_normal((9, 4096)), "bf16")
    tr, _ = half_tensor(rng.standard_normal((9, 4096)), "bf16")
    tw, _ = half_tensor(rng.standard_normal(4096), "bf16")
    fn = mq.rmsnorm_fp8 if fp8 else mq.rmsnorm_int8
    out = fn(tx, tw, EPS, residual=tr)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn(tx, tw, EPS, residual=tr, out=out[0], s_out=out[1], h_out=out[2])
    for _ in range(3):
        tx.copy_(half_tensor(rng.standard_normal((9, 4096)), "bf16")[0])
        want = fn(tx, tw, EPS, residual=tr)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want))
