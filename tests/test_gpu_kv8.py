"""The paged e4m3 KV cache on an MI355X: appends bit-exact against the oracle
(every byte of the cache, the ones that must not change too), attention within
the bound derived for its arithmetic (``oracle.fp8.kv8_attention_bound``) for
single tokens and prompts, every page size and head layout, lengths around
every tile's border, NaN codes behind the last token, empty rows, unknown
pages, caches past 4 GB, graph replays with changing lengths."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import fp8 as o8
from tests.fp8_util import codes_of, codes_tensor, half_tensor, random_codes
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu


def _up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _dt(half):
    import torch
    return torch.bfloat16 if half == "bf16" else torch.float16


def _table(rng, totals, page, P, width=None):
    """Tables of distinct pages in no order; unused entries hold numbers that
    would fault if they were followed."""
    need = [-(-t // page) for t in totals]
    width = width or max(1, max(need))
    ids = rng.permutation(P)[:sum(need)]
    t = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, P], size=(len(totals), width)).astype(np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


def _cache(rng, P, H, page, D):
    """Any byte may stand anywhere before a token is written: NaN codes too."""
    return (rng.integers(0, 256, (P, H, page, D), dtype=np.uint8), rng.integers(0, 256, (P, H, D, page), dtype=np.uint8),
            np.exp2(rng.integers(-9, -4, (P, H))).astype(np.float32), np.exp2(rng.integers(-9, -4, (P, H))).astype(np.float32))


def _fill(rng, cache, table, totals):
    """Finite codes for every token that the sequences hold (normal values)."""
    kc, vc, _, _ = cache
    P, H, page, D = kc.shape
    for b, total in enumerate(totals):
        for t0 in range(0, total, page):
            p, n = table[b, t0 // page], min(page, total - t0)
            if not 0 <= p < P:
                continue
            kc[p, :, :n] = o8.e4m3_encode(np.clip(rng.standard_normal((H, n, D)) * 90, -448, 448))
            vc[p, :, :, :n] = o8.e4m3_encode(np.clip(rng.standard_normal((H, D, n)) * 90, -448, 448))


def _dev_cache(cache):
    return codes_tensor(cache[0]), codes_tensor(cache[1]), _up(cache[2]), _up(cache[3])


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _check_append(rng, news, totals, H, D, page, half, what, k=None, v=None, cache=None, table=None, max_q=None):
    P = sum(-(-t // page) for t in totals) + 3
    cache = cache or _cache(rng, P, H, page, D)
    P = cache[0].shape[0]
    table = _table(rng, totals, page, P) if table is None else table
    # older tokens hold finite codes (a page's older codes may move)
    olds = [max(t - n, 0) for n, t in zip(news, totals)]
    if k is None:
        _fill(rng, cache, table, olds)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    lens = np.array(totals, np.int32)
    T = int(cu[-1])
    amp = np.exp2(rng.uniform(-6, 4, (T, H, 1)))
    tk, kf = half_tensor(rng.standard_normal((T, H, D)) * amp if k is None else k, half)
    tv, vf = half_tensor(rng.standard_normal((T, H, D)) * amp if v is None else v, half)
    announce(f"kv8_append {what} {half} H={H} D={D} page={page} new={news[:4]} total={totals[:4]}")
    dev = _dev_cache(cache)
    mq.kv8_append(tk, tv, *dev, _up(table), _up(cu), _up(lens), max_q_len=max_q or max(max(news), 1))
    want = o8.kv8_append_ref(kf, vf, *cache, table, cu, lens)
    for name, a, b in (("k", dev[0], want[0]), ("v", dev[1], want[1])):
        bad = np.argwhere(codes_of(a) != b)
        assert bad.size == 0, f"{what}: {len(bad)} {name} codes differ, first at {bad[:3].tolist()}"
    for name, a, b in (("k", dev[2], want[2]), ("v", dev[3], want[3])):
        assert np.array_equal(host(a).view(np.uint32), b.view(np.uint32)), f"{what}: {name} scales differ"
    return want, table


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_bitexact(page, D, half):
    rng = np.random.default_rng(page + D)
    _check_append(rng, [1, 1, 1], [1, page, page + 1], 2, D, page, half, "one token")
    _check_append(rng, [5, 1, 0, 37], [5, 200, 90, 37 + 3], 3, D, page, half, "a few")
    _check_append(rng, [page, 2 * page, page - 1, page + 1], [page, 2 * page + 7, 4 * page - 1, 3 * page], 1, D, page,
                  half, "whole pages")
    _check_append(rng, [700], [1000], 2, D, page, half, "prompt")


def test_append_in_steps_moves_scales():
    """One token at a time with growing, falling and zero values: every step
    against the oracle on the cache the step before left."""
    rng = np.random.default_rng(1)
    cache, table = None, np.array([[2, 0, 3]], np.int32)
    for step in range(40):
        amp = [1.0, 0.0, 1e-4, 30.0, 2.0, 500.0, 0.3][step % 7] * (1 + step)
        k = rng.standard_normal((1, 2, 64)) * amp
        if cache is None:
            cache = _cache(rng, 4, 2, 16, 64)
        cache, _ = _check_append(rng, [1], [step + 1], 2, 64, 16, "bf16", f"step {step}", k=k, v=-k[:, ::-1],
                                 cache=cache, table=table)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
def test_append_extremes(half):
    """Scale borders (amax of 448 2^e and one step above), zeros, the smallest
    and largest values of the type, signed zeros, exact ties of codes."""
    rng = np.random.default_rng(2)
    big, tiny = (65504.0, 6e-8) if half == "fp16" else (3.38e38, 1e-40)
    above = 448 * (1 + 2.0 ** -10) if half == "fp16" else 450.0
    rows = [448.0, above, 224.0, big, tiny, 0.0, 1.75, 17.0]
    T = len(rows)
    k = np.zeros((T, 1, 64))
    for t, a in enumerate(rows):
        k[t, 0] = a * np.resize([1.0, -0.5, 0.0, -0.0, 1 / 16, 17 / 448, 19 / 448], 64)
    for n in range(T):  # every row in a page of its own
        _check_append(rng, [1], [1], 1, 64, 16, half, f"amax {rows[n]}", k=k[n:n + 1], v=k[n:n + 1])
    _check_append(rng, [T], [T], 1, 64, 16, half, "together", k=k, v=k)


def test_append_strided_slices_and_padding():
    """k and v as slices of one projection's output, rows behind the last
    sequence present: the same bytes as dense copies."""
    import torch
    rng = np.random.default_rng(3)
    H, D, page, Hq = 2, 128, 32, 8
    news, totals = [3, 1, 40], [3, 77, 51]
    T = sum(news)
    fused, _ = half_tensor(rng.standard_normal((T + 5, (Hq + 2 * H) * D)), "bf16")
    k = fused[:, Hq * D:(Hq + H) * D].view(T + 5, H, D)
    v = fused[:, (Hq + H) * D:].view(T + 5, H, D)
    cache = _cache(rng, 12, H, page, D)
    table = _table(rng, totals, page, 12)
    _fill(rng, cache, table, [t - n for n, t in zip(news, totals)])
    cu, lens = np.concatenate([[0], np.cumsum(news)]).astype(np.int32), np.array(totals, np.int32)
    a, b = _dev_cache(cache), _dev_cache(cache)
    announce("kv8_append strided")
    mq.kv8_append(k, v, *a, _up(table), _up(cu), _up(lens), max_q_len=64)
    mq.kv8_append(k[:T].contiguous(), v[:T].contiguous(), *b, _up(table), _up(cu), _up(lens), max_q_len=40)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    want = o8.kv8_append_ref(k.float().cpu().numpy(), v.float().cpu().numpy(), *cache, table, cu, lens)
    assert np.array_equal(codes_of(a[0]), want[0]) and np.array_equal(codes_of(a[1]), want[1])


def test_append_unknown_pages_and_short_lengths():
    """Page numbers that are not of the pool, tokens past the table, more new
    tokens than the sequence holds, no tokens at all: skipped, nothing else
    touched."""
    rng = np.random.default_rng(4)
    table = np.array([[1, -1, 2], [9, 3, 5], [4, 0, 2 ** 31 - 1]], np.int32)
    cache = _cache(rng, 6, 2, 16, 64)
    k = rng.standard_normal((48 + 20 + 7, 2, 64))
    _check_append(rng, [48, 20, 7], [48, 20, 4], 2, 64, 16, "fp16", "unknown pages", k=k, v=k, cache=cache, table=table)
    cache = _cache(rng, 6, 2, 16, 64)
    _check_append(rng, [10, 30], [0, 70], 2, 64, 16, "fp16", "past the table", k=k[:40], v=k[:40], cache=cache,
                  table=np.array([[1], [2]], np.int32))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _check_attention(rng, news, totals, Hkv, G, D, page, half, what, qamp=1.0, cache=None, table=None, scale=None,
                     width=None, pad=0):
    import torch
    P = sum(-(-t // page) for t in totals) + 3
    if cache is None:
        cache = _cache(rng, P, Hkv, page, D)
    P = cache[0].shape[0]
    if table is None:
        table = _table(rng, totals, page, P, width)
        _fill(rng, cache, table, totals)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(cu[-1]) + pad
    tq, qf = half_tensor(rng.standard_normal((T, Hkv * G, D)) * qamp, half)
    scale = D ** -0.5 if scale is None else scale
    announce(f"kv8_attention {what} {half} Hkv={Hkv} G={G} D={D} page={page} new={news[:5]} total={totals[:5]}")
    out = torch.full((T, Hkv * G, D), 7.0, dtype=_dt(half), device="cuda")
    args = _up(table), _up(cu), _up(np.array(totals, np.int32))
    got = mq.kv8_attention(tq, *_dev_cache(cache), *args, max_q_len=max(max(news), 1), softmax_scale=scale, out=out)
    got = host(got.float()).astype(np.float64)
    o64, mag, sub = o8.kv8_attention_ref(qf, *cache, table, cu, totals, scale)
    none = np.isnan(o64)
    assert np.all(got[none] == 7.0), f"{what}: rows of no sequence changed"
    bound = o8.kv8_attention_bound(qf, 448.0 * float(cache[2].max()), scale, D, max(max(totals), 1), o64, mag, sub, half)
    over = np.where(none, 0.0, np.abs(got - o64) / bound)
    assert np.all(over <= 1.0), (f"{what}: worst err/bound {np.nanmax(over):.3g} at "
                                 f"{np.unravel_index(np.nanargmax(over), over.shape)}")
    assert not np.isnan(over).any()
    return got


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_lengths(page, D, half):
    rng = np.random.default_rng(page * D)
    _check_attention(rng, [1] * len(LENS), LENS, 2, 4, D, page, half, "decode lengths")


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16, 17, 32])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_decode_head_layouts(Hkv, G):
    rng = np.random.default_rng(G * 10 + Hkv)
    _check_attention(rng, [1, 1, 1], [300, 1, 77], Hkv, G, 128, 64, "bf16", "head layouts")


@pytest.mark.parametrize("news", [[2, 1, 3], [5, 5, 0], [16, 1, 2], [8, 8, 8]])
def test_few_new_tokens(news):
    rng = np.random.default_rng(sum(news))
    _check_attention(rng, news, [max(n, 1) + t for n, t in zip(news, (0, 62, 500))], 2, 4, 128, 32, "fp16", "few tokens")


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_prompts(page, D, half):
    rng = np.random.default_rng(page + D + 1)
    _check_attention(rng, [100, 1, 64, 65], [100, 50, 200, 65], 2, 4, D, page, half, "prompts")


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_prompts_in_wide_tables(page, D, half):
    """Tables for 64 K tokens: what they could hold decides for the prompt form
    and many splits, most of them without keys."""
    rng = np.random.default_rng(page + D + 2)
    _check_attention(rng, [100, 1, 64, 65], [100, 50, 200, 65], 2, 4, D, page, half, "wide", width=65536 // page)
    _check_attention(rng, [90, 0, 30], [40, 0, 0], 2, 3, D, page, half, "wide, empty rows", pad=2, width=65536 // page)
    _check_attention(rng, [300], [2111], 1, 5, D, page, half, "wide, longer", qamp=6.0, width=65536 // page)


@pytest.mark.parametrize("news,totals,G", [([1030, 999], [1030, 1500], 8), ([513, 200, 777], [1100, 200, 2000], 4)])
def test_prompts_large(news, totals, G):
    """Large enough for the prompt form by what they hold."""
    rng = np.random.default_rng(G)
    _check_attention(rng, news, totals, 4, G, 128, 64, "bf16", "large")


@pytest.mark.parametrize("G", [1, 3, 8])
def test_prompt_long(G):
    rng = np.random.default_rng(G)
    _check_attention(rng, [513, 200], [1100, 200], 1, G, 128, 64, "bf16", "long prompts")


def test_prompts_of_many_sequences():
    """More sequences than a wavefront has lanes, some without new tokens, some
    of several row tiles."""
    rng = np.random.default_rng(18)
    news = [int(n) for n in rng.integers(0, 30, 150)]
    news[0], news[70], news[149] = 0, 300, 200
    totals = [n + int(t) for n, t in zip(news, rng.integers(0, 60, 150))]
    _check_attention(rng, news, totals, 1, 4, 64, 16, "bf16", "many sequences", pad=2)


@pytest.mark.parametrize("page", [16, 128])
def test_prompts_over_many_tiles(page):
    """Workgroups that walk thousands of keys: 64 row tiles, so the keys are
    hardly split, over up to 54 tiles of 64 with unknown pages among them."""
    rng = np.random.default_rng(19)
    totals = [3400, 2111]
    table = _table(rng, totals, page, 400)
    cache = _cache(rng, 400, 8, page, 64)
    _fill(rng, cache, table, totals)
    table[0, 1100 // page] = table[1, 2000 // page] = -1
    _check_attention(rng, [66, 300], totals, 8, 32, 64, page, "fp16", "many tiles", cache=cache, table=table)


def test_empty_rows_and_padding():
    """No key at all, more new tokens than cached ones, rows of no sequence."""
    rng = np.random.default_rng(7)
    _check_attention(rng, [1, 1, 1], [0, 5, 0], 2, 4, 128, 16, "bf16", "empty decode", pad=3)
    _check_attention(rng, [4, 2], [2, 0], 2, 4, 64, 16, "fp16", "few empty", pad=1)
    _check_attention(rng, [90, 30], [40, 0], 2, 4, 128, 32, "bf16", "empty prompt rows", pad=2)


def test_unknown_pages_count_for_nothing():
    rng = np.random.default_rng(8)
    for news, G in (([1, 1], 4), ([70, 3], 2)):
        totals = [150, 75]
        table = np.array([[3, -1, 5, 1, 99, 2, 7, 8, 9, 10], [4, 2 ** 31 - 1, 6, 0, -7, 0, 0, 0, 0, 0]], np.int32)
        cache = _cache(rng, 11, 2, 16, 128)
        _fill(rng, cache, table, totals)
        _check_attention(rng, news, totals, 2, G, 128, 16, "bf16", "unknown pages", cache=cache, table=table)


def test_unknown_pages_in_prompts():
    rng = np.random.default_rng(21)
    totals = [150, 75]
    table = np.full((2, 4096), -1, np.int32)
    table[:, :10] = [[3, -1, 5, 1, 99, 2, 7, 8, 9, 10], [4, 2 ** 31 - 1, 6, 0, -7, 0, 0, 0, 0, 0]]
    cache = _cache(rng, 11, 2, 16, 128)
    _fill(rng, cache, table[:, :10], totals)
    _check_attention(rng, [90, 3], totals, 2, 2, 128, 16, "bf16", "unknown pages, prompt form", cache=cache, table=table)


@pytest.mark.parametrize("news", [[250], [200, 70]])
def test_wide_scales_in_prompts(news):
    """As the next test, through the prompt form."""
    rng = np.random.default_rng(22)
    totals = [900, 333][:len(news)]
    for what, qamp, klo, vlo in (("wide v", 1.0, -8, -30), ("peaked", 12.0, -6, -12), ("wide v and peaked", 8.0, -6, -30)):
        P = 100
        cache = _cache(rng, P, 2, 16, 128)
        cache = (cache[0], cache[1], np.exp2(rng.integers(klo, -4, (P, 2))).astype(np.float32),
                 np.exp2(rng.integers(vlo, 6, (P, 2))).astype(np.float32))
        table = _table(rng, totals, 16, P, 4096)
        _fill(rng, cache, table, totals)
        _check_attention(rng, news, totals, 2, 4, 128, 16, "bf16", what, qamp=qamp, cache=cache, table=table)


@pytest.mark.parametrize("news", [[1, 1], [80, 70]])
def test_wide_scales_and_peaked_scores(news):
    """V scales of neighbouring pages far apart and scores that leave one token
    nearly alone: the weight that counts may sit in the page of the smallest
    scale."""
    rng = np.random.default_rng(9)
    totals = [900, 333]
    for what, qamp, klo, vlo in (("wide v", 1.0, -8, -30), ("peaked", 12.0, -6, -12), ("wide v and peaked", 8.0, -6, -30)):
        P = 100
        cache = _cache(rng, P, 2, 16, 128)
        cache = (cache[0], cache[1], np.exp2(rng.integers(klo, -4, (P, 2))).astype(np.float32),
                 np.exp2(rng.integers(vlo, 6, (P, 2))).astype(np.float32))
        table = _table(rng, totals, 16, P)
        _fill(rng, cache, table, totals)
        _check_attention(rng, news, totals, 2, 4, 128, 16, "bf16", what, qamp=qamp, cache=cache, table=table)


def test_scales_that_are_no_powers_of_two():
    rng = np.random.default_rng(10)
    cache = _cache(rng, 60, 2, 32, 128)
    cache = (cache[0], cache[1], rng.uniform(1e-3, 1e-2, (60, 2)).astype(np.float32),
             rng.uniform(1e-3, 1e-2, (60, 2)).astype(np.float32))
    table = _table(rng, [1000, 700], 32, 60)
    _fill(rng, cache, table, [1000, 700])
    _check_attention(rng, [1, 1], [1000, 700], 2, 4, 128, 32, "fp16", "any scales", cache=cache, table=table)


@pytest.mark.parametrize("news", [[1], [300]])
def test_split_keys(news):
    """One long sequence: its keys are split over workgroups; a table far wider
    than the sequence splits a short one too."""
    rng = np.random.default_rng(11)
    _check_attention(rng, news, [9001], 1, 4, 128, 64, "bf16", "long")
    _check_attention(rng, news, [700], 1, 4, 64, 16, "fp16", "wide table", width=4096)
    _check_attention(rng, news, [0], 1, 4, 64, 16, "fp16", "wide table, nothing cached", width=4096)


@pytest.mark.parametrize("tiles", [9, 17, 65, 66, 67, 129, 133, 261])
def test_every_number_of_splits(tiles):
    """From two to all of the splits, odd numbers too; the last key alone in its
    tile. Beside it a short sequence, whose splits are mostly without keys."""
    rng = np.random.default_rng(tiles)
    _check_attention(rng, [1], [64 * tiles - 63], 1, 2, 64, 64, "bf16", f"{tiles} tiles", qamp=3.0)
    _check_attention(rng, [1, 1], [64 * tiles - 63, 70], 1, 4, 128, 32, "fp16", f"{tiles} tiles and two", qamp=3.0)


def test_one_query_row_is_its_value():
    """A sequence of one token: the output is that token's value, rounded once."""
    rng = np.random.default_rng(12)
    cache = _cache(rng, 3, 2, 16, 128)
    table = np.array([[1]], np.int32)
    cache[0][1, :, 0] = random_codes(rng, (2, 128))
    cache[1][1, :, :, 0] = random_codes(rng, (2, 128))
    got = _check_attention(rng, [1], [1], 2, 3, 128, 16, "bf16", "one token", cache=cache, table=table)
    want = o8.e4m3_decode(cache[1][1, :, :, 0]) * cache[3][1][:, None].astype(np.float64)
    assert np.array_equal(got.reshape(2, 3, 128), np.repeat(want[:, None], 3, 1))  # exact: 4 bits times a power of two


@pytest.mark.parametrize("D", [64, 128])
def test_many_short_sequences(D):
    """From 128 workgroups on, sequences of up to 16 tiles of keys go unsplit
    over eight wavefronts."""
    rng = np.random.default_rng(D + 20)
    totals = [int(n) for n in rng.integers(1, 1025, 66)]
    totals[0], totals[1], totals[2] = 1024, 1, 961
    _check_attention(rng, [1] * 66, totals, 2, 4, D, 32, "bf16", "many short")


def test_cache_past_four_gigabytes():
    """Pages whose byte offsets pass 2^32: append and both attention forms, at
    the far end of a pool whose other pages are never written."""
    import torch
    H, D, page, P = 8, 128, 64, 70000  # 4.6 GB of K codes, as many of V
    kc = torch.empty((P, H, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.empty((P, H, D, page), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks, vs = torch.ones((P, H), device="cuda"), torch.ones((P, H), device="cuda")
    rng = np.random.default_rng(13)
    ids = np.array([P - 1, 3, P - 2], np.int32)
    total = 150
    table = _up(ids[None])
    tk, kf = half_tensor(rng.standard_normal((total, H, D)), "bf16")
    tv, vf = half_tensor(rng.standard_normal((total, H, D)), "bf16")
    lens = _up(np.array([total], np.int32))
    announce("kv8 past 4 GB: append")
    mq.kv8_append(tk, tv, kc, vc, ks, vs, table, _up(np.array([0, total], np.int32)), lens, max_q_len=total)
    small = (np.zeros((3, H, page, D), np.uint8), np.zeros((3, H, D, page), np.uint8), np.ones((3, H), np.float32),
             np.ones((3, H), np.float32))
    want = o8.kv8_append_ref(kf, vf, *small, np.array([[0, 1, 2]], np.int32), [0, total], [total])
    at = torch.from_numpy(ids).long().cuda()
    tail = total % page
    gk, gv = codes_of(kc.view(torch.uint8)[at]), codes_of(vc.view(torch.uint8)[at])
    assert np.array_equal(gk[:2], want[0][:2]) and np.array_equal(gv[:2], want[1][:2])
    assert np.array_equal(gk[2, :, :tail], want[0][2, :, :tail]) and np.array_equal(gv[2, :, :, :tail], want[1][2, :, :, :tail])
    for n in (1, 100):
        tq, qf = half_tensor(rng.standard_normal((n, 4 * H, D)), "bf16")
        cu = np.array([0, n], np.int32)
        announce(f"kv8 past 4 GB: attention of {n}")
        got = host(mq.kv8_attention(tq, kc, vc, ks, vs, table, _up(cu), lens, max_q_len=n).float())
        o64, mag, sub = o8.kv8_attention_ref(qf, *want, np.array([[0, 1, 2]]), cu, [total], D ** -0.5)
        bound = o8.kv8_attention_bound(qf, 448.0 * float(want[2].max()), D ** -0.5, D, total, o64, mag, sub, "bf16")
        assert np.all(np.abs(got - o64) <= bound)


@pytest.mark.parametrize("new", [1, 40])
def test_graph_replays_with_changing_lengths(new):
    """Append and attention captured once with static buffers; between replays
    the lengths, tables and inputs change. Every replay equals the eager calls
    on a second cache, bit for bit."""
    import torch
    rng = np.random.default_rng(14)
    B, H, G, D, page, P, width = 3, 2, 4, 128, 16, 400, 100
    T = B * new
    a = _dev_cache(_cache(rng, P, H, page, D))
    for t in a[:2]:
        t.view(torch.uint8).zero_()
    b = tuple(t.clone() for t in a)
    table = _up(rng.permutation(P)[:B * width].reshape(B, width).astype(np.int32))
    cu = _up((np.arange(B + 1) * new).astype(np.int32))
    lens = torch.full((B,), new, dtype=torch.int32, device="cuda")
    q, _ = half_tensor(rng.standard_normal((T, H * G, D)), "bf16")
    kv, _ = half_tensor(rng.standard_normal((T, 2, H, D)), "bf16")
    out = torch.empty_like(q)
    need = mq.kv8_attention_workspace_bytes(T, B, H * G, H, D, page, width, new)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step(cache, o, w):
        mq.kv8_append(kv[:, 0], kv[:, 1], *cache, table, cu, lens, max_q_len=new)
        mq.kv8_attention(q, *cache, table, cu, lens, max_q_len=new, out=o, workspace=w)

    announce(f"kv8 graph, {new} new tokens")
    step(tuple(t.clone() for t in a), out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, out, ws)
    for r in range(4):
        lens.copy_(torch.tensor([new * (r + 1), min(1600, new + 500 * r), new + r], dtype=torch.int32))
        q.copy_(half_tensor(rng.standard_normal((T, H * G, D)), "bf16")[0])
        kv.copy_(half_tensor(rng.standard_normal((T, 2, H, D)) * (1 + 3 * r), "bf16")[0])
        eager = torch.empty_like(out)
        step(b, eager, None)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"replay {r}"
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b)), f"replay {r}: cache"


def test_other_stream_and_strided_queries():
    import torch
    rng = np.random.default_rng(15)
    H, G, D, page = 2, 4, 128, 64
    totals, news = [500, 130, 64], [1, 1, 1]
    cache = _cache(rng, 20, H, page, D)
    table = _table(rng, totals, page, 20)
    _fill(rng, cache, table, totals)
    fused, _ = half_tensor(rng.standard_normal((3, (H * G + 2 * H) * D)), "fp16")
    q = fused[:, :H * G * D].view(3, H * G, D)
    args = (*_dev_cache(cache), _up(table), _up(np.array([0, 1, 2, 3], np.int32)), _up(np.array(totals, np.int32)))
    want = mq.kv8_attention(q.contiguous(), *args, max_q_len=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mq.kv8_attention(q, *args, max_q_len=1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_empty_batches():
    import torch
    cache = _dev_cache(_cache(np.random.default_rng(0), 2, 2, 16, 64))
    i32 = dict(dtype=torch.int32, device="cuda")
    none = torch.empty((0, 3), **i32), torch.zeros((1,), **i32), torch.empty((0,), **i32)
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    assert mq.kv8_attention(q, *cache, *none, max_q_len=1).shape == (0, 4, 64)
    mq.kv8_append(q[:, :2], q[:, :2], *cache, *none, max_q_len=1)
