"""Pins of the e4m3 cache's oracle: what is not finite in an append."""

import numpy as np

from oracle import fp8 as o


def test_append_of_what_is_not_finite():
    # one page of 4 tokens, one head, three dimensions; the older token holds NaN
    kc, vc = np.zeros((1, 1, 4, 3), np.uint8), np.zeros((1, 1, 3, 4), np.uint8)
    kc[0, 0, 0] = vc[0, 0, :, 0] = [0xFF, 0x38, 0x7F]  # NaN, 1, NaN
    ks, vs = np.ones((1, 1), np.float32), np.ones((1, 1), np.float32)
    x = np.float32([[[np.inf, 896.0, np.nan]], [[-np.inf, 2.0, 4.0]]])
    a = o.kv8_append_ref(x, x, kc, vc, ks, vs, np.zeros((1, 1), np.int32), [0, 2], [3])
    assert a[2][0, 0] == 2.0 and a[3][0, 0] == 2.0  # 896 decides, not the infinity
    for codes in (a[0][0, 0], a[1][0, 0].T):
        assert codes[0].tolist() == [0xFF, 0x30, 0x7F]  # 0.5: moved to the new scale; NaN as it was
        assert codes[1].tolist() == [0x7F, 0x7E, 0x7F]
        assert codes[2].tolist() == [0x7F, 0x38, 0x40]
        assert not codes[3].any()
    y = np.float32([[[np.nan, np.inf, -np.inf]]])
    b = o.kv8_append_ref(y, y, kc, vc, ks, vs, np.zeros((1, 1), np.int32), [0, 1], [1])
    assert b[2][0, 0] == np.float32(2.0 ** -100) and b[0][0, 0, 0].tolist() == [0x7F] * 3
