"""Pins of the e4m3 oracle: the format against torch's, hand-worked values, and
the definitions against brute force."""

import numpy as np
import pytest

from oracle import fp8 as o


def test_decode_against_torch():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(o.e4m3_decode(codes), want, equal_nan=True)
    assert o.e4m3_decode(np.uint8(0x7E)) == 448.0 and o.e4m3_decode(np.uint8(0x01)) == 2.0 ** -9


def test_encode_against_torch_and_ties():
    import torch
    rng = np.random.default_rng(0)
    grid = o.e4m3_decode(np.arange(127, dtype=np.uint8))
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64),
                        rng.uniform(-448, 448, 5000).astype(np.float32),
                        (rng.standard_normal(5000) * 0.01).astype(np.float32)])
    v = np.concatenate([v, -v]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o.e4m3_encode(v), want)
    # 17 lies between 16 and 18 and goes to 16 (even), 19 to 20
    assert o.e4m3_decode(o.e4m3_encode([17.0, 19.0])).tolist() == [16.0, 20.0]


def test_round_half_against_torch():
    import torch
    rng = np.random.default_rng(1)
    v = (rng.standard_normal(4000) * np.exp2(rng.uniform(-20, 10, 4000))).astype(np.float32)
    for half, dt in (("fp16", torch.float16), ("bf16", torch.bfloat16)):
        assert np.array_equal(o.round_half(v, half), torch.from_numpy(v).to(dt).float().numpy())


def test_rmsnorm_hand_row():
    v, h = o.rmsnorm_ref(np.float32([[3.0, 4.0, 0.0, 0.0]]), np.float32([1, 2, 1, 1]), 0.0, half="fp16")
    # mean of squares 6.25, root 2.5
    assert np.array_equal(h, [[3, 4, 0, 0]])
    r = np.float32(0.4)
    assert np.array_equal(v, np.float32([[np.float32(3) * r, np.float32(np.float32(4) * r) * 2, 0, 0]]))


def test_quant_blocks_properties():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((5, 300)).astype(np.float32)
    v[3, 128:256] = 0
    q, s = o.quant_fp8_blocks_ref(v)
    assert s.shape == (3, 5) and s[1, 3] == 0 and not q[3, 128:256].any()
    for b in range(3):
        part = o.e4m3_decode(q[:, 128 * b:128 * (b + 1)]) * s[b][:, None].astype(np.float64)
        x = v[:, 128 * b:128 * (b + 1)].astype(np.float64)
        # half a step of the value, or of the smallest normal code
        assert np.all(np.abs(part - x) <= 2.0 ** -4 * np.abs(x) * (1 + 2.0 ** -20) + 2.0 ** -10 * s[b][:, None] * 1.001)
        assert np.all((np.max(np.abs(o.e4m3_decode(q[:, 128 * b:128 * (b + 1)])), axis=1) == 448) | (s[b] == 0))


def test_mm_brute_force():
    rng = np.random.default_rng(3)
    M, N, K = 3, 130, 144
    xq = rng.integers(0, 127, (M, K)).astype(np.uint8)
    wq = (rng.integers(0, 127, (N, K)) | (rng.integers(0, 2, (N, K)) << 7)).astype(np.uint8)
    sx, sw = rng.random((2, M)).astype(np.float32), rng.random((2, 2)).astype(np.float32)
    y, mag = o.fp8_mm_ref(xq, sx, wq, sw)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        acc = 0.0
        for k in range(K):
            acc += float(o.e4m3_decode(xq[m, k])) * float(sx[k // 128, m]) * float(o.e4m3_decode(wq[n, k])) * float(
                sw[n // 128, k // 128])
        assert abs(acc - y[m, n]) <= 1e-12 * mag[m, n]


@pytest.mark.parametrize("amax,want", [(448.0, 0), (448.5, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (0.0, -100),
                                       (1e-40, -100), (3.3e38, 120)])
def test_page_scale(amax, want):
    assert o.page_scale(np.float32(amax)) == np.float32(2.0) ** want


def test_append_grows_and_keeps():
    # one page of 4 tokens, one head, two dimensions
    kc = np.zeros((2, 1, 4, 2), np.uint8)
    vc = np.zeros((2, 1, 2, 4), np.uint8)
    ks, vs = np.full((2, 1), 7.0, np.float32), np.full((2, 1), 7.0, np.float32)
    table = np.array([[1]], np.int32)
    x = np.float32([[[448.0, -3.0]]])
    a = o.kv8_append_ref(x, x, kc, vc, ks, vs, table, [0, 1], [1])
    assert a[2][1, 0] == 1.0 and a[2][0, 0] == 7.0  # a fresh page's old scale does not count
    assert o.e4m3_decode(a[0][1, 0, 0]).tolist() == [448, -3] and o.e4m3_decode(a[1][1, 0, :, 0]).tolist() == [448, -3]
    big = np.float32([[[1000.0, 1.0]]])
    b = o.kv8_append_ref(big, big, *a, table, [0, 1], [2])
    assert b[2][1, 0] == 4.0
    assert o.e4m3_decode(b[0][1, 0, :2]).tolist() == [[112, -0.75], [256, 0.25]]  # 250 is between 240 and 256
    small = np.float32([[[0.5, 0.5]]])
    c = o.kv8_append_ref(small, small, *b, table, [0, 1], [3])
    assert c[2][1, 0] == 4.0 and o.e4m3_decode(c[1][1, 0, :, 2]).tolist() == [0.125, 0.125]


def test_attention_hand_cases():
    rng = np.random.default_rng(4)
    P, H, page, D = 3, 2, 4, 8
    kc = rng.integers(0, 100, (P, H, page, D)).astype(np.uint8)
    vc = rng.integers(0, 100, (P, H, D, page)).astype(np.uint8)
    ks, vs = np.full((P, H), 0.5, np.float32), np.full((P, H), 2.0, np.float32)
    table = np.array([[2, 0], [1, -1]], np.int32)
    q = rng.standard_normal((4, 4, D)).astype(np.float32)
    o64, mag, _ = o.kv8_attention_ref(q, kc, vc, ks, vs, table, [0, 2, 3], [2, 0], 0.3)
    # the first query of sequence 0 sees one token: its value, whatever the scores
    assert np.allclose(o64[0, 1], o.e4m3_decode(vc[2, 0, :, 0]) * 2.0, rtol=1e-12)
    # the second: two tokens by hand
    k = o.e4m3_decode(kc[2, 1, :2]) * 0.5
    s = k @ q[1, 3].astype(np.float64) * 0.3
    w = np.exp(s - s.max())
    w /= w.sum()
    assert np.allclose(o64[1, 3], w @ (o.e4m3_decode(vc[2, 1, :, :2]).T * 2.0), rtol=1e-12)
    assert not o64[2].any() and np.isnan(o64[3]).all()  # nothing cached; no sequence's row
    # a page that is not in the pool counts for nothing
    a, _, _ = o.kv8_attention_ref(q[:1], kc, vc, ks, vs, table[1:], [0, 1], [6], 0.3)
    b, _, _ = o.kv8_attention_ref(q[:1], kc, vc, ks, vs, table[1:, :1], [0, 1], [4], 0.3)
    assert np.allclose(a, b, rtol=1e-12)
