"""Pins of the drafted tokens' oracle on the CPU: rotation against complex
multiplication, trees by hand, verification against the distribution that it has
to draw from, the cache's clean-up by hand."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import drafts as od
from oracle import fp8 as o8


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 2, 64)).astype(np.float32), np.array([0, 3, 1, 2, 3])
    ang = rng.uniform(0, 6, (4, 16))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    got = od.rotate_ref(x, pos, cs, interleaved=interleaved)
    assert np.array_equal(got[..., 32:], x[..., 32:])
    z = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) if interleaved else (x[..., :16] + 1j * x[..., 16:32])
    z = z * np.exp(1j * ang[pos])[:, None]
    want = np.empty((5, 2, 32))
    if interleaved:
        want[..., 0::2], want[..., 1::2] = z.real, z.imag
    else:
        want[..., :16], want[..., 16:] = z.real, z.imag
    # two products and a sum of values below 6, the table's rounding as much again
    assert np.abs(got[..., :32] - want).max() < 5 * 6 * 2.0 ** -24 * 2
    assert np.isnan(od.rotate_ref(x, np.array([4, -1, 0, 0, 0]), cs)[:2, :, :32]).all()


def test_norm_before_rotation():
    x = np.full((1, 1, 32), 3.0, np.float32)
    cs = np.concatenate([np.ones((1, 8)), np.zeros((1, 8))], 1).astype(np.float32)
    w = np.linspace(0.5, 2, 32).astype(np.float32)
    got = od.rotate_ref(x, np.array([0]), cs, w, eps=0.0)
    assert np.allclose(got[0, 0], w, rtol=2.0 ** -22)


def test_tree_by_hand():
    #   0 - 1 - 3      a second sequence of one node; node 4 hangs on nothing valid
    #     \ 2 - 5
    parents = np.array([-1, 0, 0, 1, 7, 2, -1])
    words, pos = od.tree_ref(parents, np.array([0, 6, 7]), np.array([16, 9]), 2)
    assert words[:, 0].tolist() == [1, 3, 5, 11, 16, 37, 1] and not words[:, 1].any()
    assert pos.tolist() == [10, 11, 11, 12, 10, 12, 8]


def test_tree_words_cross():
    words, pos = od.tree_ref(np.arange(-1, 69), np.array([0, 70]), np.array([70]), 3)
    assert words[69].view(np.uint32).tolist() == [2 ** 32 - 1, 2 ** 32 - 1, 63] and pos[69] == 69
    assert words[31].view(np.uint32).tolist() == [2 ** 32 - 1, 0, 0]


def _first_tokens(probs, tokens, parents, draft, grid):
    """How often each token follows node 0, over a grid of uniform numbers for all
    nodes (the middle of every cell: exact but for cells that a border cuts)."""
    V, n = probs.shape[1], len(tokens)
    u = (np.arange(grid) + 0.5) / grid
    seen = np.zeros(V)
    for cell in np.ndindex(*(grid,) * n):
        kept, path, nxt = od.verify_ref(probs, tokens, u[list(cell)].astype(np.float32), np.array([0, n]), n, parents, draft)
        seen[tokens[path[0, 1]] if kept[0] > 1 else nxt[0]] += 1
    return seen / grid ** n


def test_verification_draws_from_the_target():
    """Trees (two siblings, one of them again with the same token) and chains with
    the draft's probabilities: the first token after the root has the root's
    distribution. A border cuts at most one cell of each of the n axes."""
    p = np.array([[0.5, 0.25, 0.125, 0.125], [0.25, 0.25, 0.25, 0.25], [0.1, 0.2, 0.3, 0.4], [0, 0, 1, 0]], np.float32)
    got = _first_tokens(p, np.array([9, 2, 0, 2]), np.array([-1, 0, 0, 0]), None, 16)
    assert np.abs(got - p[0]).max() <= 4 / 16
    got = _first_tokens(p[:3], np.array([9, 1, 0]), np.array([-1, 0, 0]), None, 32)
    assert np.abs(got - p[0]).max() <= 3 / 32
    q = np.array([0.125, 0.5, 0.25, 0.125], np.float32)
    total = np.zeros(4)
    for x in range(4):  # the draft draws x with q(x)
        total += q[x] * _first_tokens(p[:2], np.array([9, x]), None, np.stack([q, q]), 64)
    assert np.abs(total - p[0]).max() <= 2 / 64


def test_verification_by_hand():
    p = np.array([[0.5, 0.5, 0, 0], [0, 0.25, 0.75, 0], [0, 0, 0, 1]], np.float32)
    u = np.array([0.5, 0.25, 0.9], np.float32)
    kept, path, nxt = od.verify_ref(p, np.array([0, 1, 2]), u, np.array([0, 3]), 4)
    assert kept.tolist() == [2] and path.tolist() == [[0, 1, -1, -1]]
    assert nxt.tolist() == [1]  # token 2 of row 1 was rejected (0.9 >= 0.75): what is left is token 1
    assert od.verify_ref(p, np.array([0, 1, 2]), np.float32([0.5, 0.25, 0.7]), np.array([0, 3]), 4)[0].tolist() == [3]
    # nothing left of the row after its only token was rejected: the row itself
    one = np.array([[0, 1, 0, 0]] * 2, np.float32)
    assert od.verify_ref(one, np.array([0, 1]), np.float32([0.0, 1.0]), np.array([0, 2]), 2)[2].tolist() == [1]


def test_which_tests_of_a_draft_are_exact():
    """Products of two binary32 values have 48 bits: exact in binary64. What rejected
    siblings leave, and its product, are rounded: 2^-54 a term, 2^-53 of the product."""
    rng = np.random.default_rng(4)
    u, q = rng.random((2, 500)).astype(np.float32).astype(np.float64)
    assert all(Fraction(a * b) == Fraction(a) * Fraction(b) for a, b in zip(u, q))
    rounded = 0
    for i in range(500):
        p = (rng.dirichlet(np.ones(6))[:5]).astype(np.float32).astype(np.float64)
        left, exact = 1.0, Fraction(1)
        for k, x in enumerate(p):
            left, exact = left - x, exact - Fraction(x)
            assert abs(Fraction(left) - exact) <= (k + 1) * Fraction(1, 2 ** 54)
        got = u[i] * left
        assert abs(Fraction(got) - Fraction(u[i]) * Fraction(left)) <= Fraction(got) / 2 ** 53
        rounded += Fraction(got) != Fraction(u[i]) * exact
    assert rounded > 0  # one is enough: such a test cannot be called exact


def test_norm_factor_next_to_a_rounding_border():
    """The factor of two orders of the sum differs by 2^-46 of itself at most, and so
    by one step of binary32 only where a border lies that near."""
    rng = np.random.default_rng(5)
    for _ in range(300):
        x = (rng.standard_normal(128) * np.exp2(rng.integers(-12, 8, 128))).astype(np.float16).astype(np.float64)
        want = sum(Fraction(v) ** 2 for v in x) / 128 + Fraction(1e-6)
        for order in (np.arange(128), rng.permutation(128)):
            total = 0.0
            for v in x[order]:
                total += v * v
            r = 1.0 / np.sqrt(total / 128 + 1e-6)
            assert abs(Fraction(r) ** 2 * want - 1) <= Fraction(1, 2 ** 45)


def test_keep_by_hand():
    page, D = 16, 64
    kc = np.zeros((1, 3, 1, page, D), np.uint8)
    vc = np.zeros((1, 3, 1, D, page), np.uint8)
    ks, vs = np.full((1, 3, 1), 0.25, np.float32), np.full((1, 3, 1), 0.25, np.float32)
    ks[0, 1] = 1.0
    code = lambda v: o8.e4m3_encode(np.full(D, float(v)))
    kc[0, 0, 0, 14], kc[0, 0, 0, 15], kc[0, 1, 0, 1], kc[0, 0, 0, 3] = code(1), code(2), code(448), code(8)
    vc[0, 0, 0, :, 14], vc[0, 1, 0, :, 1] = code(1), code(5)
    table, cu, lens = np.array([[0, 1]]), np.array([0, 4]), np.array([18])
    out = od.keep_ref(kc, vc, ks, vs, table, cu, lens, np.array([[0, 3, -1, -1]]), np.array([2]))
    assert out[2][0, 0, 0] == 1.0 and out[3][0, 0, 0] == 0.25  # 448 needs the larger scale, 5 does not
    assert np.array_equal(out[0][0, 0, 0, 15], code(448)) and np.array_equal(out[1][0, 0, 0, :, 15], code(5))
    assert np.array_equal(out[0][0, 0, 0, 14], code(0.25)) and np.array_equal(out[0][0, 0, 0, 3], code(2))
    assert np.array_equal(out[0][0, 1], kc[0, 1])


def test_tree_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(3)
    q = rng.standard_normal((5, 2, 64)).astype(np.float32)
    from tests.kv8_util import paged
    cache, table = paged(rng, [40], 1, 16, 64)
    cu, lens = np.array([0, 5]), np.array([40])
    words, _ = od.tree_ref(np.arange(-1, 4), cu, lens, 1)
    a = o8.kv8_attention_rows(q, *cache, table, cu, lens, 0.125, "fp16")
    b = o8.kv8_attention_rows(q, *cache, table, cu, lens, 0.125, "fp16", tree=words)
    assert np.array_equal(a[0], b[0]) and np.allclose(a[1], b[1], rtol=1e-3)
