"""Plain CPU definitions of the e4m3 operators (test infrastructure, as
``oracle.ref``): RMS norm with 8-bit output, the e4m3 quantizer and product
with a scale per block of 128, the paged e4m3 KV cache and attention over it.

16-bit inputs are passed as float32 arrays of the values; ``half`` names their
format ("fp16" or "bf16") where a result is rounded back to it. e4m3 values
are uint8 codes (OCP: exponent bias 7, largest 448, no infinities, 0x7F NaN).
"""

import numpy as np

E4M3_MAX = 448.0
BLOCK = 128
MIN_SCALE_EXP, MAX_SCALE_EXP = -100, 120


def e4m3_decode(codes):
    """uint8 codes -> float64 values."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


_GRID = e4m3_decode(np.arange(127, dtype=np.uint8))  # 0 .. 448, ascending


def e4m3_encode(values):
    """Finite values within +-448 -> nearest codes, ties to the even code (as
    the grid's neighbours differ by one code, even means an even mantissa)."""
    v = np.asarray(values, dtype=np.float64)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_GRID, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def round_half(values, half):
    """float32 values -> nearest fp16 / bf16 values (ties to even), as float32."""
    v = np.asarray(values, dtype=np.float32)
    if half == "fp16":
        return v.astype(np.float16).astype(np.float32)
    b = v.view(np.uint32).astype(np.uint64)
    return ((((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16) & 0xFFFFFFFF).astype(np.uint32).view(np.float32)


def rmsnorm_ref(x, weight, eps, residual=None, half="fp16"):
    """(v, h): h = rne16(x + residual), v = fl32(fl32(h * r) * w) with
    r = fl32(1 / sqrt(mean(h^2) + eps)), the mean and root in float64."""
    h = np.asarray(x, np.float32)
    if residual is not None:
        h = round_half(h + np.asarray(residual, np.float32), half)
    ms = np.sum(h.astype(np.float64) ** 2, axis=1) / h.shape[1]
    r = (1.0 / np.sqrt(ms + eps)).astype(np.float32)
    return (h * r[:, None]) * np.asarray(weight, np.float32)[None, :], h


def quant_fp8_blocks_ref(v):
    """float32 [M, K] -> (codes uint8 [M, K], s_x float32 [ceil(K/128), M])."""
    v = np.asarray(v, np.float32)
    M, K = v.shape
    nb = -(-K // BLOCK)
    q = np.zeros((M, K), np.uint8)
    s = np.zeros((nb, M), np.float32)
    for b in range(nb):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        a = np.max(np.abs(part), axis=1)
        s[b] = np.divide(a, np.float32(E4M3_MAX), dtype=np.float32)
        nz = s[b] > 0
        quot = np.divide(part[nz], s[b][nz, None], dtype=np.float32)
        q[nz, b * BLOCK:(b + 1) * BLOCK] = e4m3_encode(np.clip(quot, -E4M3_MAX, E4M3_MAX))
    return q, s


def fp8_mm_ref(xq, s_x, wq, s_w):
    """(y64, mag): the product in float64 and the sum of the terms' magnitudes."""
    M, K = xq.shape
    N = wq.shape[0]
    kb, nb = np.arange(K) // BLOCK, np.arange(N) // BLOCK
    x = e4m3_decode(xq) * s_x.astype(np.float64).T[:, kb]
    w = e4m3_decode(wq) * s_w.astype(np.float64)[nb][:, kb]
    return x @ w.T, np.abs(x) @ np.abs(w).T


def fp8_mm_bound(y64, mag, gmax, K, half):
    """Largest |y - y64| of the kernel's arithmetic.

    The fp8 matrix unit aligns the products of 8 consecutive k to the largest
    exponent among them and drops what lies below 2^-13 of it, so each of the
    other 7 products errs by less than 2^-13 of the largest: 7 2^-13 gmax with
    gmax the sum over the groups of their largest product. The groups' sums, a
    block's scale product and multiply-add and the ranges' sums are binary32:
    at most 16 groups and 4 more steps a block and 16 ranges of 2^-23 of the
    terms' magnitude each. Then the output's rounding."""
    u = 2.0 ** -8 if half == "bf16" else 2.0 ** -11
    steps = 20 + -(-K // BLOCK) + 16
    err = 7 * 2.0 ** -13 * gmax + steps * 2.0 ** -23 * mag
    return u * (np.abs(y64) + err) + err + (2.0 ** -25 if half == "fp16" else 2.0 ** -133)


def page_scale(amax):
    """Smallest power of two s with amax <= 448 s, its exponent in [-100, 120]."""
    amax = np.asarray(amax, np.float64)
    e = np.ceil(np.log2(np.maximum(amax, 2.0 ** -140) / E4M3_MAX))
    # log2 is not exact next to a border: settle it by the definition
    e = np.where(amax <= E4M3_MAX * 2.0 ** (e - 1), e - 1, e)
    e = np.where(amax > E4M3_MAX * 2.0 ** e, e + 1, e)
    return (2.0 ** np.clip(e, MIN_SCALE_EXP, MAX_SCALE_EXP)).astype(np.float32)


def kv8_append_ref(k, v, k_cache, v_cache, k_scales, v_scales, table, cu, lens):
    """The cache after the append (copies): k, v float32 [T, H, D]; k_cache
    uint8 [P, H, page, D], v_cache [P, H, D, page], scales [P, H]."""
    kc, vc, ks, vs = k_cache.copy(), v_cache.copy(), k_scales.copy(), v_scales.copy()
    P, H, page, D = kc.shape
    width = table.shape[1]
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        for pos0 in range((max(start, 0) // page) * page, int(lens[b]), page):
            slot = pos0 // page
            if slot >= width or not 0 <= table[b, slot] < P or n <= 0:
                continue
            p = int(table[b, slot])
            lo, hi = max(start, pos0), min(int(lens[b]), pos0 + page)
            if lo >= hi or lo < 0:
                continue
            rows = slice(int(cu[b]) + lo - start, int(cu[b]) + hi - start)
            for h in range(H):
                for x, c, s, tr in ((k, kc, ks, False), (v, vc, vs, True)):
                    new = np.asarray(x[rows, h], np.float32)
                    tile = c[p, h].T if tr else c[p, h]  # [page, D] view
                    odd = ~np.isfinite(new)  # counts for no scale, becomes the NaN code
                    new = np.where(odd, np.float32(0), new)
                    scale = page_scale(np.max(np.abs(new)))
                    if lo > pos0:
                        old = s[p, h]
                        if scale > old:
                            had = tile[:lo - pos0].copy()
                            nan = (had & 0x7F) == 0x7F
                            moved = e4m3_decode(np.where(nan, 0, had)) * np.float64(np.float32(old / scale))
                            tile[:lo - pos0] = np.where(nan, had, e4m3_encode(np.clip(moved, -E4M3_MAX, E4M3_MAX)))
                        else:
                            scale = old
                    codes = e4m3_encode(np.clip(new.astype(np.float64) / np.float64(scale), -E4M3_MAX, E4M3_MAX))
                    tile[lo - pos0:hi - pos0] = np.where(odd, np.uint8(0x7F), codes)
                    s[p, h] = scale
    return kc, vc, ks, vs


def _seen(pos, row0, n, L, tree):
    """[n, len(pos)] truth values: which positions the n rows from row0 on, the last
    of L tokens, see: those up to their own, or with words `tree` [T, W] every one
    before the new tokens and of these the ones with a bit in the row's words."""
    if tree is None:
        return pos[None, :] <= (L - n + np.arange(n))[:, None]
    j = pos - (L - n)
    w = np.clip(j // 32, 0, tree.shape[1] - 1)
    bits = (tree[row0:row0 + n].astype(np.int64)[:, w] >> (j % 32)[None, :]) & 1
    return (j < 0)[None, :] | ((bits == 1) & (j < 32 * tree.shape[1])[None, :])


def kv8_attention_ref(q, k_cache, v_cache, k_scales, v_scales, table, cu, lens, scale, tree=None):
    """(o64 [T, Hq, D], mag, sub): attention of q (float32 [T, Hq, D]) in
    float64; mag = sum_t p_t |v_t| and sub = max_t(p_t s_v,t) sum_t |code_t|,
    the terms of the error bound. Rows that see nothing are 0; rows of no
    sequence are NaN."""
    T, Hq, D = q.shape
    P, H, page, _ = k_cache.shape
    G = Hq // H
    o = np.full((T, Hq, D), np.nan)
    mag, sub = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        o[int(cu[b]):int(cu[b + 1])] = 0.0
        L = max(0, min(L, table.shape[1] * page))
        if n <= 0 or L <= 0:
            continue
        pos = np.arange(L)
        ids = table[b, pos // page]
        good = (ids >= 0) & (ids < P)
        ids = np.where(good, ids, 0)
        for h in range(H):
            kk = e4m3_decode(k_cache[ids, h, pos % page]) * k_scales[ids, h].astype(np.float64)[:, None]
            vcode = e4m3_decode(v_cache[ids, h, :, pos % page])
            sv = v_scales[ids, h].astype(np.float64)
            for g in range(G):
                qq = q[int(cu[b]):int(cu[b + 1]), h * G + g].astype(np.float64)
                s = qq @ np.where(good[:, None], kk, 0.0).T * scale
                seen = _seen(pos, int(cu[b]), n, int(lens[b]), tree) & good[None, :]
                s = np.where(seen, s, -np.inf)
                top = np.max(s, axis=1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                tot = p.sum(1, keepdims=True)
                p = p / np.where(tot > 0, tot, 1.0)
                vv = np.where(good[:, None], vcode * sv[:, None], 0.0)
                rows = slice(int(cu[b]), int(cu[b + 1]))
                o[rows, h * G + g] = p @ vv
                mag[rows, h * G + g] = p @ np.abs(vv)
                sub[rows, h * G + g] = np.max(p * sv[None, :], axis=1)[:, None] * np.sum(
                    np.abs(np.where(good[:, None], vcode, 0.0)), axis=0)[None, :]
    return o, mag, sub


def kv8_attention_bound(q, k_absmax, scale, D, length, o64, mag, sub, half):
    """Largest |o - o64| of the kernel's arithmetic, element by element.

    score: D exact products summed in binary32 (2^-23 each, as the matrix unit
    may truncate), two scalings and the exponent's argument (2^-24 each): with
    S = sum |q k| scale <= max|q| max|k| D scale an error of
    ds <= (D + 4) 2^-23 S, which moves a weight by the factor exp(+-ds), the
    largest score the same again. exp2 and log2 err by 2^-22 of themselves and
    an exponent of up to 2^8 by 2^-16. A weight is rounded to fp16 (2^-11, or
    2^-25 of the largest weight below fp16's normal range: the `sub` term);
    sums of `length` weights and products 2^-23 each step."""
    u = 2.0 ** -8 if half == "bf16" else 2.0 ** -11
    S = float(np.max(np.abs(q))) * k_absmax * D * abs(scale)
    ds = (D + 4) * 2.0 ** -23 * S
    rel = 2.0 ** -11 + 4 * ds + 2.0 ** -14 + 2 * length * 2.0 ** -23
    err = rel * mag + 2.0 ** -25 * sub
    return u * (np.abs(o64) + err) + err + (2.0 ** -25 if half == "fp16" else 2.0 ** -133)


def kv8_attention_rows(q, k_cache, v_cache, k_scales, v_scales, table, cu, lens, scale, half, tree=None):
    """(o64, bound): ``kv8_attention_ref``'s output and the largest |o - o64| of
    the kernel's arithmetic, row by row from what the row sees.

    With S = max_t scale sum_d |q_d k_td| and V = max_t |log2 v_scale| over the
    keys of the row, and T their tiles of 64:
    - a score sums D products in binary32, 2^-23 of their magnitude each; its
      factor has four roundings of 2^-24, the multiply-add, the reference and the
      difference to it three more of 2^-24 of at most 2 (log2(e) S + V) + 16, the
      logarithm errs by 2^-22 of V. An exponent (base 2) is off by at most
        d = 2^-23 ((D + 8) log2(e) S + 4 V + 16)
      which moves a weight by ln 2 d of itself, the sum of the weights likewise;
    - a weight is rounded to fp16 (2^-11 of itself; the largest weight of a row is
      2^11 or more, so one too small for fp16's normal range is off by 2^-25, at
      most 2^-36 of the largest: `sub`); the sum is of unrounded ones;
    - exp2 errs by 2^-22, where the reference moves all sums by as much again;
      the matrix unit adds eight groups of 8 products per tile, each addition off
      by 2^-23 of the sum; parts of wavefronts and splits join with fewer than 100
      more: 2^-23 (12 T + 128) in all;
    - the output is rounded once (2^-11, bf16 2^-8 of itself)."""
    T, Hq, D = q.shape
    P, H, page, _ = k_cache.shape
    o64, mag, sub = kv8_attention_ref(q, k_cache, v_cache, k_scales, v_scales, table, cu, lens, scale, tree)
    rel = np.zeros((T, Hq, 1))
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        length = max(0, min(L, table.shape[1] * page))
        if n <= 0 or length <= 0:
            continue
        pos = np.arange(length)
        ids = table[b, pos // page]
        good = (ids >= 0) & (ids < P)
        ids = np.where(good, ids, 0)
        seen = _seen(pos, int(cu[b]), n, L, tree) & good[None, :]
        last = L - n + np.arange(n) if tree is None else np.full(n, length)
        tiles = np.clip(last, 0, length) // 64 + 1
        for hq in range(Hq):
            h = hq // (Hq // H)
            k = np.abs(e4m3_decode(k_cache[ids, h, pos % page])) * k_scales[ids, h].astype(np.float64)[:, None]
            s = np.abs(q[int(cu[b]):int(cu[b + 1]), hq].astype(np.float64)) @ np.where(good[:, None], k, 0.0).T * abs(scale)
            S = np.max(np.where(seen, s, 0.0), axis=1)
            with np.errstate(divide="ignore", invalid="ignore"):
                V = np.max(np.where(seen, np.abs(np.log2(v_scales[ids, h].astype(np.float64)))[None, :], 0.0), axis=1)
            d = 2.0 ** -23 * ((D + 8) * np.log2(np.e) * S + 4 * V + 16)
            rel[int(cu[b]):int(cu[b + 1]), hq, 0] = 2.0 ** -11 + 2 * np.log(2) * d + 2.0 ** -23 * (12 * tiles + 128)
    u = 2.0 ** -8 if half == "bf16" else 2.0 ** -11
    err = 1.01 * (rel * mag + 2.0 ** -36 * sub)
    return o64, u * (np.abs(o64) + err) + err + (2.0 ** -25 if half == "fp16" else 2.0 ** -133)
