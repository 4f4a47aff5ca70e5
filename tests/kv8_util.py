"""Caches and checks of the attention tests that look at single rows."""

import numpy as np

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import codes_of, codes_tensor, half_tensor
from tests.gpu_util import announce, host


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def empty_cache(P, H, page, D, scale=2.0 ** -6):
    """Codes 0 everywhere, one scale."""
    return (np.zeros((P, H, page, D), np.uint8), np.zeros((P, H, D, page), np.uint8),
            np.full((P, H), scale, np.float32), np.full((P, H), scale, np.float32))


def put(cache, table, b, t, k=None, v=None):
    """Codes k, v [H, D] (or [D], for every head) of token t of sequence b."""
    page = cache[0].shape[2]
    p = table[b, t // page]
    if k is not None:
        cache[0][p, :, t % page] = k
    if v is not None:
        cache[1][p, :, :, t % page] = v


def random_codes(rng, shape):
    return o8.e4m3_encode(np.clip(rng.standard_normal(shape) * 90, -448, 448))


def paged(rng, totals, Hkv, page, D, width=None, spare=1):
    """(cache, table) for sequences of `totals` tokens and `spare` more: random
    pages, numbers of no pool where none is needed, codes of normal values, NaN
    codes in pages of no sequence."""
    need = [-(-(t + spare) // page) for t in totals]
    P = sum(need) + 2
    cache = empty_cache(P, Hkv, page, D)
    cache[0][:], cache[1][:] = 0x7F, 0xFF
    table = np.full((len(totals), width or max(need)), 2 ** 31 - 1, np.int32)
    ids = rng.permutation(P)
    for b, n in enumerate(need):
        table[b, :n], ids = ids[:n], ids[n:]
        at = table[b, :n]
        cache[0][at], cache[1][at] = random_codes(rng, (n, Hkv, page, D)), random_codes(rng, (n, Hkv, D, page))
    for s in cache[2:]:
        s[:] = np.exp2(rng.integers(-9, -5, (P, Hkv)))
    return cache, table


def planted(rng, news, totals, Hkv, G, D, page, width=None):
    """(q, cache, table): peaked softmax where the last key that a row sees has
    its largest score, and the key behind it, which it does not see, a larger one
    still: a row that loses the one or takes the other is far off."""
    cache, table = paged(rng, totals, Hkv, page, D, width)
    cache[2][:] = 2.0 ** -3
    cache[0][(cache[0] & 0x7F) != 0x7F] = 0  # score 0 but for the planted ones
    q = np.empty((sum(news), Hkv * G, D))
    at = 0
    for b, (n, L) in enumerate(zip(news, totals)):
        if n == 0:
            continue
        way = rng.choice([-1.0, 1.0], (Hkv, D))
        q[at:at + n] = np.repeat(way, G, axis=0) * rng.uniform(0.5, 1.5, (n, Hkv * G, 1))
        at += n
        for i in range(n + 1):  # the last one: behind the sequence
            put(cache, table, b, L - n + i, k=o8.e4m3_encode(way * (3 + 0.25 * i) / 2.0 ** -3))
    return q, cache, table


def counted(rng, news, totals, Hkv, G, D, page, width=None, half="bf16"):
    """(q, cache, table, want) for softmax_scale = 0: every key that a row sees
    weighs the same, and token t of kv head h holds 1 in dimension (t + 7 h) % D
    alone, so that the output counts keys."""
    cache, table = paged(rng, totals, Hkv, page, D, width)
    cache[3][:] = 1.0
    dims = np.arange(D)
    for b, total in enumerate(totals):
        for t in range(total):
            put(cache, table, b, t, v=np.stack([np.where(dims == (t + 7 * h) % D, 0x38, 0) for h in range(Hkv)]))
    want = np.zeros((sum(news), Hkv * G, D))
    at = 0
    for n, L in zip(news, totals):
        for i in range(n):
            sees = max(L - n + i + 1, 0)
            for h in range(Hkv):
                if sees:
                    want[at + i, h * G:(h + 1) * G] = np.bincount((np.arange(sees) + 7 * h) % D, minlength=D) / sees
        at += n
    return rng.standard_normal((sum(news), Hkv * G, D)), cache, table, want


def append(k, v, half, cache, table, news, totals, what):
    """kv8_append on a copy of a host cache, every byte against the oracle: the
    cache after it."""
    cu, lens = np.concatenate([[0], np.cumsum(news)]).astype(np.int32), np.array(totals, np.int32)
    (tk, kf), (tv, vf) = half_tensor(k, half), half_tensor(v, half)
    announce(f"kv8_append {what} {half} {cache[0].shape} new={news[:5]} total={totals[:5]}")
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    mq.kv8_append(tk, tv, *dev, up(table), up(cu), up(lens), max_q_len=max(news))
    got = codes_of(dev[0]), codes_of(dev[1]), host(dev[2]), host(dev[3])
    want = o8.kv8_append_ref(kf, vf, *cache, table, cu, lens)
    for name, a, b in zip(("K codes", "V codes", "K scales", "V scales"), got, want):
        bad = np.argwhere(a != b)
        assert bad.size == 0, f"{what}: {len(bad)} {name} differ, first at {bad[:3].tolist()}"
    return got


def attend(tq, cache, table, cu, lens, what, scale=None, most=None):
    """kv8_attention of q over a host cache, into rows that hold 7: float64 values."""
    import torch
    announce(f"kv8_attention {what} {tq.dtype} q={tuple(tq.shape)} new={np.diff(cu)[:5].tolist()} total={list(lens)[:5]}")
    out = torch.full(tq.shape, 7.0, dtype=tq.dtype, device="cuda")
    mq.kv8_attention(tq, codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3]), up(table),
                     up(np.asarray(cu, np.int32)), up(np.asarray(lens, np.int32)),
                     max_q_len=most or max(1, int(np.max(np.diff(cu)))), softmax_scale=scale, out=out)
    return host(out.float()).astype(np.float64)


def check_rows(q, half, cache, table, cu, lens, what, scale=None, fro=None):
    """The call within the rows' own bounds and, where `fro` is given, every
    sequence within that relative Frobenius error."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    tq, qf = half_tensor(q, half)
    got = attend(tq, cache, table, cu, lens, what, scale)
    o64, bound = o8.kv8_attention_rows(qf, *cache, table, cu, lens, scale, half)
    none = np.isnan(o64)
    assert np.all(got[none] == 7.0), f"{what}: rows of no sequence changed"
    over = np.where(none, 0.0, np.abs(got - o64) / bound)
    assert not np.isnan(over).any(), f"{what}: NaN in row {np.argwhere(np.isnan(over))[0].tolist()}"
    assert np.all(over <= 1.0), f"{what}: worst err/bound {over.max():.3g} at {np.unravel_index(over.argmax(), over.shape)}"
    for b in range(len(lens)):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        size = np.linalg.norm(o64[rows])
        if fro and size > 0:
            rel = np.linalg.norm(got[rows] - o64[rows]) / size
            assert rel <= fro, f"{what}: sequence {b} of {lens[b]} keys, relative Frobenius error {rel:.3g}"
    return got
