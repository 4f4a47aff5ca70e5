"""Append with rotation and head norms on an MI355X: q, every byte of the cache
and every scale bit-exact against the oracle, for both kinds of pairs, whole and
partial rotations, positions given and not, strided and in-place rows, NaN and
positions outside the table, rows and pages that must stay as they are."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from oracle import drafts as od
from oracle import fp8 as o8
from tests.draft_util import offsets, table_of_angles
from tests.fp8_util import codes_of, codes_tensor, half_tensor
from tests.gpu_util import announce, host
from tests.kv8_util import paged, up

pytestmark = pytest.mark.gpu


def _cache(rng, news, totals, H, page, D, width=None):
    """Older tokens' codes are finite, everything else may hold anything."""
    cache, table = paged(rng, [max(t, 1) for t in totals], H, page, D, width)
    return cache, table


def _place(news, totals):
    return np.concatenate([np.arange(t - n, t) for n, t in zip(news, totals)] or [np.zeros(0)]).astype(np.int64)


def check(rng, news, totals, Hq, H, D, page, half, what, rot=None, norm=False, nxt=False, positions=None, max_pos=None,
          pad=0, cache=None, table=None, most=None, fused=False, in_place=False, amp=1.0, values=None):
    import torch
    rot = rot or D
    if cache is None:
        cache, table = _cache(rng, news, totals, H, page, D)
    cu, lens = offsets(news), np.array(totals, np.int32)
    T, used = int(cu[-1]) + pad, int(cu[-1])
    heads = Hq + 2 * H
    x = rng.standard_normal((T, heads, D)) * amp * np.exp2(rng.uniform(-4, 4, (T, 1, 1))) if values is None else values
    t, xf = half_tensor(x, half)
    cs = table_of_angles(rng, max_pos or max(max(totals), 1), rot)
    pos = _place(news, totals) if positions is None else np.asarray(positions[:used], np.int64)
    w = [half_tensor(rng.uniform(0.5, 1.5, D), half) for _ in "qk"] if norm else [(None, None)] * 2
    if fused or in_place:
        q, k, v = t.split([Hq, H, H], 1)
    else:
        q, k, v = (s.contiguous() for s in t.split([Hq, H, H], 1))
    out = q if in_place else torch.full((T, Hq, D), 7.0, dtype=t.dtype, device="cuda")
    announce(f"kv8_rope_append {what} {half} Hq={Hq} H={H} D={D} page={page} rot={rot} norm={norm} next={nxt} "
             f"new={news[:4]} total={totals[:4]}")
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    tp = None if positions is None else up(np.asarray(positions, np.int32))
    before = t.clone()
    got = mq.kv8_rope_append(q, k, v, *dev, up(table), up(cu), up(lens), max_q_len=most or max(max(news), 1),
                             cos_sin=up(cs), positions=tp, q_weight=w[0][0], k_weight=w[1][0], eps=1e-5, interleaved=nxt,
                             out=out)
    assert got.data_ptr() == out.data_ptr()
    with np.errstate(all="ignore"):
        qr = o8.round_half(od.rotate_ref(xf[:used, :Hq], pos, cs, w[0][1], 1e-5, nxt), half)
        kr = od.rotate_ref(xf[:used, Hq:Hq + H], pos, cs, w[1][1], 1e-5, nxt)
        want = o8.kv8_append_ref(kr, xf[:used, Hq + H:], *cache, table, cu, lens)
    gq = host(got.float())
    same = (gq[:used] == qr) | (np.isnan(gq[:used]) & np.isnan(qr))
    assert same.all(), f"{what}: {np.sum(~same)} of q differ, first at {np.argwhere(~same)[:3].tolist()}"
    rest = before[used:, :Hq].float().cpu().numpy() if in_place else 7.0
    assert np.all(gq[used:] == rest), f"{what}: rows of no sequence changed"
    if in_place:
        assert torch.equal(t[:, Hq:].view(torch.int16), before[:, Hq:].view(torch.int16)), f"{what}: k or v changed"
    for name, a, b in (("K", dev[0], want[0]), ("V", dev[1], want[1])):
        bad = np.argwhere(codes_of(a) != b)
        assert bad.size == 0, f"{what}: {len(bad)} {name} codes differ, first at {bad[:3].tolist()}"
    for name, a, b in (("K", dev[2], want[2]), ("V", dev[3], want[3])):
        assert np.array_equal(host(a).view(np.uint32), b.view(np.uint32)), f"{what}: {name} scales differ"


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_lengths(page, D, half):
    rng = np.random.default_rng(page + D)
    check(rng, [1, 1, 1], [1, page, page + 1], 4, 2, D, page, half, "one token")
    check(rng, [5, 1, 0, 37], [5, 200, 90, 40], 3, 3, D, page, half, "a few", norm=True)
    check(rng, [page, 2 * page, page - 1, page + 1], [page, 2 * page + 7, 4 * page - 1, 3 * page], 5, 1, D, page, half,
          "whole pages", nxt=True)
    check(rng, [700], [1000], 4, 2, D, page, half, "prompt", norm=True, rot=D // 2)


@pytest.mark.parametrize("nxt", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 80), (128, 112), (128, 128)])
def test_rotations(D, rot, norm, nxt):
    rng = np.random.default_rng(rot + D)
    check(rng, [3, 20], [10, 20], 6, 2, D, 16, "bf16", "rotations", rot=rot, norm=norm, nxt=nxt)
    check(rng, [3, 20], [10, 20], 6, 2, D, 64, "fp16", "rotations", rot=rot, norm=norm, nxt=nxt)


@pytest.mark.parametrize("Hq,H", [(1, 1), (7, 1), (12, 4), (32, 8), (40, 5)])
def test_head_layouts(Hq, H):
    rng = np.random.default_rng(Hq)
    check(rng, [1, 9, 2], [40, 9, 17], Hq, H, 128, 16, "fp16", "heads", norm=True)


@pytest.mark.parametrize("fused,in_place", [(True, False), (True, True)])
@pytest.mark.parametrize("nxt", [False, True])
def test_slices_and_in_place(fused, in_place, nxt):
    rng = np.random.default_rng(4)
    for half, page, news in (("bf16", 32, [3, 1, 40]), ("fp16", 128, [300, 1]), ("bf16", 16, [1, 1])):
        totals = [n + t for n, t in zip(news, (0, 76, 11))]
        check(rng, news, totals, 8, 2, 128, page, half, "slices", norm=True, nxt=nxt, fused=fused, in_place=in_place, pad=3,
              most=max(news) + 5)


def test_positions_of_a_tree():
    rng = np.random.default_rng(5)
    news, totals = [26, 7], [90, 40]
    pos = np.concatenate([64 + np.minimum(np.arange(26), 5), 33 + np.array([0, 1, 1, 2, 2, 2, 3]), [-9, 10 ** 6]])
    for nxt in (False, True):
        check(rng, news, totals, 4, 2, 64, 32, "fp16", "tree", positions=pos, nxt=nxt, pad=2)


def test_positions_outside_the_table():
    """NaN for the rotated part, in q and as K codes; the token counts for no scale."""
    rng = np.random.default_rng(6)
    pos = [-1, 5, 20, 2 ** 31 - 1, -2 ** 31, 19]
    for rot in (32, 64):
        for norm in (False, True):
            check(rng, [6], [30], 2, 2, 64, 16, "bf16", "outside", rot=rot, norm=norm, positions=pos, max_pos=20)
    # more new tokens than cached ones: the first stand before position 0
    check(rng, [6, 3], [4, 0], 2, 1, 64, 16, "fp16", "before the first", max_pos=20)


@pytest.mark.parametrize("half", ["fp16", "bf16"])
def test_values_that_are_not_finite_and_extremes(half):
    rng = np.random.default_rng(7)
    big = 65504.0 if half == "fp16" else 3e38
    x = rng.standard_normal((9, 4, 64))
    x[1, :, 5], x[2, :, 40], x[3, :, 0], x[4] = np.inf, np.nan, -np.inf, 0.0
    x[5] *= 1e-7
    x[6, :, ::3] = big
    x[7, :, ::2] = -0.0
    for norm in (False, True):
        for nxt in (False, True):
            check(rng, [9], [20], 2, 1, 64, 16, half, "not finite", values=x, norm=norm, nxt=nxt)


def test_unknown_pages_skip_keys_only():
    rng = np.random.default_rng(8)
    cache, table = _cache(rng, [20, 5], [60, 20], 2, 16, 128)
    table[0, 3], table[1, 1] = -1, 2 ** 31 - 1
    check(rng, [20, 5], [60, 20], 4, 2, 128, 16, "bf16", "unknown pages", cache=cache, table=table)
    check(rng, [20, 5], [60, 20], 4, 2, 128, 16, "bf16", "narrow table", cache=cache, table=table[:, :3].copy())


def test_many_sequences():
    rng = np.random.default_rng(9)
    news = [int(n) for n in rng.integers(0, 4, 70)]
    totals = [n + int(t) for n, t in zip(news, rng.integers(0, 50, 70))]
    check(rng, news, totals, 4, 1, 64, 16, "bf16", "many", norm=True, pad=1)


def test_growing_scales_step_by_step():
    rng = np.random.default_rng(10)
    import torch  # noqa: F401
    totals, news, H, D = [1], [1], 1, 64
    cache, table = _cache(rng, [1], [48], H, 16, D)
    for step, amp in enumerate([1.0, 0.0, 1e-4, 30.0, 2.0, 500.0, 0.3, 4000.0, 1.0] * 2):
        check(rng, news, [step + 1], 2, H, D, 16, "bf16", f"step {step}", cache=cache, table=table, amp=amp)
        x, xf = half_tensor(rng.standard_normal((1, H, D)) * amp, "bf16")
        cache = o8.kv8_append_ref(xf, xf, *cache, table, np.array([0, 1], np.int32), np.array([step + 1], np.int32))


def test_agrees_with_the_plain_append():
    """A table of cosine 1 and sine 0 changes nothing: the bytes of kv8_append."""
    import torch
    rng = np.random.default_rng(11)
    news, totals, H, D, page = [1, 50, 3], [33, 50, 70], 2, 128, 32
    cache, table = _cache(rng, news, totals, H, page, D)
    x, _ = half_tensor(rng.standard_normal((54, 3 * H, D)), "fp16")
    q, k, v = x.split([H, H, H], 1)
    cs = up(np.concatenate([np.ones((80, 64)), np.zeros((80, 64))], 1).astype(np.float32))
    b = up(table), up(offsets(news)), up(np.array(totals, np.int32))
    sides = []
    for rope in (True, False):
        dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
        if rope:
            assert torch.equal(mq.kv8_rope_append(q, k, v, *dev, *b, max_q_len=50, cos_sin=cs), q)
        else:
            mq.kv8_append(k, v, *dev, *b, max_q_len=50)
        sides.append([t.view(torch.uint8) for t in dev])
    assert all(torch.equal(s, t) for s, t in zip(*sides))


def test_rows_and_angles_past_2_31_values():
    """q, k, v and out with rows 2^26 values apart, a table of 2^24 + 40 positions:
    as with dense rows and a small table."""
    import torch
    rng = np.random.default_rng(15)
    T, Hq, H, D, page, far, max_pos = 36, 8, 2, 128, 16, 2 ** 26, 2 ** 24 + 40
    results = []
    t, _ = half_tensor(rng.standard_normal((T, Hq + 2 * H, D)), "bf16")
    cs = up(table_of_angles(rng, 40, D))
    wide = torch.zeros((T * far,), dtype=torch.bfloat16, device="cuda").view(T, far)[:, :t[0].numel()]
    wide.copy_(t.view(T, -1))
    angles = torch.zeros((max_pos, D), device="cuda")
    angles[-40:] = cs
    cache, table = _cache(rng, [T], [50], H, page, D)
    for rows, turns, pos in ((t, cs, 0), (wide.unflatten(1, t.shape[1:]), angles, max_pos - 40)):
        q, k, v = rows.split([Hq, H, H], 1)
        out = torch.zeros_like(q) if rows is t else torch.zeros(T * far, dtype=q.dtype, device="cuda").view(T, far)[:, :Hq * D].unflatten(1, (Hq, D))
        dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
        announce(f"kv8_rope_append rows {rows.stride(0)} apart, {turns.shape[0]} positions")
        mq.kv8_rope_append(q, k, v, *dev, up(table), up(np.array([0, T], np.int32)), up(np.array([50], np.int32)), T, turns,
                           positions=up(np.arange(pos, pos + T, dtype=np.int32)), out=out)
        results.append([out.clone()] + [x.view(torch.uint8).clone() for x in dev])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert results[0][0].abs().max() > 1


def test_nothing_to_do():
    import torch
    rng = np.random.default_rng(12)
    cache, table = _cache(rng, [1], [20], 2, 16, 64)
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    x = torch.zeros((0, 2, 64), dtype=torch.float16, device="cuda")
    cs = up(table_of_angles(rng, 8, 64))
    out = mq.kv8_rope_append(x, x, x, *dev, up(table), up(np.zeros(2, np.int32)), up(np.array([20], np.int32)), 1, cs)
    assert out.shape == (0, 2, 64) and np.array_equal(codes_of(dev[0]), cache[0])


def test_refusals_of_the_wrapper():
    import torch
    rng = np.random.default_rng(13)
    cache, table = _cache(rng, [2], [20], 2, 16, 64)
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    b = up(table), up(np.array([0, 2], np.int32)), up(np.array([20], np.int32))
    x = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda")
    cs, w = up(table_of_angles(rng, 30, 64)), torch.ones(64, dtype=torch.float16, device="cuda")

    def call(q=x, k=x, v=x, cs=cs, **kw):
        return mq.kv8_rope_append(q, k, v, *dev, *b, 2, cs, **kw)

    call()
    with pytest.raises(TypeError):
        call(k=x.bfloat16())
    with pytest.raises(ValueError):
        call(v=x[:1])
    with pytest.raises(ValueError):
        call(q_weight=w)
    with pytest.raises(ValueError):
        call(q_weight=w, k_weight=w[:32])
    with pytest.raises(TypeError):
        call(cs=cs.double())
    with pytest.raises(ValueError):
        call(positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(mq.MqError):
        call(cs=cs[:, :40].contiguous())
    with pytest.raises(mq.MqError):
        call(out=x[:, :, :].view(2, 2, 64), q=x.clone(), k=x)  # out over k
    with pytest.raises(ValueError):
        call(out=x.clone()[:1])
