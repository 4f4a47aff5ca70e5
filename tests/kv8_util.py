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
