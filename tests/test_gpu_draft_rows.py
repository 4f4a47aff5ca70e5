"""Drafted steps whose first sequence does not begin at row 0: rows in front of it
belong to no sequence, as those behind the last do. Every operator does what it does
without them, and leaves them alone."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from tests.draft_util import layered, offsets, random_trees, table_of_angles
from tests.fp8_util import codes_tensor, half_tensor
from tests.gpu_util import announce
from tests.kv8_util import up

pytestmark = pytest.mark.gpu

FILL = 77


def _step(news, totals, front, behind, D, page, width, G, wide):
    """The five operators one after the other -> what they wrote, caches among it."""
    import torch
    rng = np.random.default_rng(sum(news))
    Hkv, V, most, used = 2, wide, max(news), sum(news)
    cache, table = layered(rng, 1, [t + page for t in totals], Hkv, page, D, width)
    dev = [t[0].clone() for t in (codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3]))]
    parents = random_trees(rng, news, loose=0.05)
    x = rng.standard_normal((used, (G + 2) * Hkv, D))
    probs = np.exp(3 * rng.standard_normal((used, V)))
    probs = (probs / probs.sum(-1, keepdims=True)).astype(np.float32)
    tokens, uniform = rng.integers(0, V, used).astype(np.int32), rng.random(used).astype(np.float32)
    for j in range(used):  # (a child's token is often its parent's likeliest)
        tokens[j] = probs[max(j - 1, 0)].argmax() if j % 2 else tokens[j]
    angles = up(table_of_angles(rng, max(totals) + 1, D))

    def rows(a, fill):
        return np.concatenate([np.full((front, *a.shape[1:]), fill, a.dtype), a, np.full((behind, *a.shape[1:]), fill, a.dtype)])

    T = front + used + behind
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = up(table), up(offsets(news) + np.int32(front)), up(np.array(totals, np.int32))
    q, k, v = half_tensor(rows(x, 3.0), "bf16")[0].split([G * Hkv, Hkv, Hkv], 1)
    mask, pos = torch.full((T, -(-most // 32)), FILL, **i32), torch.full((T,), FILL, **i32)
    announce(f"drafted step, {front} rows in front, new={news}")
    mq.kv8_tree_mask(up(rows(parents, 0)), *batch[1:], most, mask=mask, positions=pos)
    qo, o = (torch.full((T, G * Hkv, D), float(FILL), dtype=torch.bfloat16, device="cuda") for _ in "qo")
    mq.kv8_rope_append(q, k, v, *dev, *batch, most, angles, positions=pos, out=qo)
    mq.kv8_tree_attention(qo, mask, *dev, *batch, most, out=o)
    verdict = mq.draft_verify(up(rows(probs, 0.5)), up(rows(tokens, 1)), up(rows(uniform, 0.0)), batch[1], most,
                              parents=up(rows(parents, 0)))
    mq.kv8_tree_keep(*dev, *batch, verdict[1], verdict[0])
    for t in (mask, pos, qo, o):
        assert torch.all(t[:front] == FILL) and torch.all(t[front + used:] == FILL)
    return [t[front:front + used].clone() for t in (mask, pos, qo, o)], list(verdict) + [t.view(torch.uint8) for t in dev], T


@pytest.mark.parametrize("front", [1, 37])
@pytest.mark.parametrize("news,totals,D,page,width,G,wide,form", [
    ([7, 0, 5, 1], [40, 33, 5, 200], 64, 16, None, 4, 900, "decode"),
    ([9, 3], [300, 3], 128, 64, None, 4, 40000, "decode"),
    ([90, 1, 40], [400, 20, 41], 128, 32, 2048, 4, 700, "prompt"),
    ([100] + [3] * 70, [300] + [50] * 70, 64, 16, 512, 2, 100, "prompt"),
])
def test_first_row(news, totals, D, page, width, G, wide, form, front):
    import torch
    plain = _step(news, totals, 0, 0, D, page, width, G, wide)
    moved = _step(news, totals, front, 3, D, page, width, G, wide)
    for T in (plain[2], moved[2]):
        assert mq.kv8_tree_attention_form(T, len(news), 2 * G, 2, D, page, width or -(-(max(totals) + page) // page) + 1,
                                          max(news)) == form
    for part in (0, 1):
        for a, b in zip(plain[part], moved[part]):
            assert torch.equal(a, b)
