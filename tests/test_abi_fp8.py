"""Refusals of the RMS norm and e4m3 entry points on the CPU: bad arguments are
rejected on the host before any HIP call (the pointers are fake addresses)."""

import pytest

import weight_activation_quantized_amd as mq

OK, NULL, SHAPE, ALIGN, UNSUP, WS, ALIAS, HIP = range(8)
A, B, C, D, E, F, G, H = (0x10_0000_0000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    return mq.library()


@pytest.mark.parametrize("name", ["mq_rmsnorm_int8", "mq_rmsnorm_int8_bf16", "mq_rmsnorm_fp8", "mq_rmsnorm_fp8_bf16"])
def test_rmsnorm(lib, name):
    def f(x=A, res=B, w=C, eps=1e-5, h=D, q=E, s=F, M=4, K=256):
        return getattr(lib, name)(x, res, w, eps, h, q, s, M, K, None)

    assert f(x=None) == NULL and f(w=None) == NULL and f(q=None) == NULL and f(s=None) == NULL
    assert f(res=None) == NULL and f(h=None) == NULL  # together or not at all
    assert f(M=-1) == SHAPE and f(M=1 << 22) == SHAPE
    assert f(K=8) == SHAPE and f(K=264) == SHAPE and f(K=65536 + 16) == SHAPE and f(K=0) == SHAPE
    assert f(eps=-1e-6) == UNSUP and f(eps=2.0) == UNSUP and f(eps=float("nan")) == UNSUP
    assert f(x=A + 8) == ALIGN and f(res=B + 2) == ALIGN and f(w=C + 8) == ALIGN and f(h=D + 8) == ALIGN
    assert f(q=E + 8) == ALIGN and f(s=F + 2) == ALIGN
    assert f(h=A) == ALIAS and f(h=B + 16) == ALIAS and f(q=D) == ALIAS and f(s=E + 16) == ALIAS and f(h=C) == ALIAS
    assert f(h=B, q=B + 512) == ALIAS  # in place, but the codes fall into it
    assert f(x=A, res=A, h=A) == ALIAS  # in place over x as well: x would change under its reader
    assert f(M=0) == OK and f(M=0, x=None, res=None, h=None, q=None, s=None) == OK


def test_quant_fp8(lib):
    f = lib.mq_quant_fp8_blocks
    assert f(None, B, C, 4, 256, None) == NULL and f(A, None, C, 4, 256, None) == NULL
    assert f(A, B, None, 4, 256, None) == NULL
    assert f(A, B, C, -1, 256, None) == SHAPE and f(A, B, C, 4, 250, None) == SHAPE
    assert f(A, B, C, 4, (1 << 20) + 16, None) == SHAPE and f(A, B, C, 1 << 27, 16, None) == SHAPE
    assert f(A + 8, B, C, 4, 256, None) == ALIGN and f(A, B + 8, C, 4, 256, None) == ALIGN
    assert f(A, B, C + 1, 4, 256, None) == ALIGN
    assert f(A, A + 1024, C, 4, 256, None) == ALIAS and f(A, B, B + 16, 4, 256, None) == ALIAS
    assert f(None, None, None, 0, 256, None) == OK


def test_fp8_block_mm(lib):
    def f(xq=A, sx=B, wq=C, sw=D, y=E, M=4, N=130, K=272):
        return lib.mq_fp8_block_mm(xq, sx, wq, sw, y, M, N, K, None)

    for k in ("xq", "sx", "wq", "sw", "y"):
        assert f(**{k: None}) == NULL, k
    assert f(K=8) == SHAPE and f(K=250) == SHAPE and f(K=(1 << 20) + 16) == SHAPE
    assert f(M=-1) == SHAPE and f(N=-1) == SHAPE and f(N=(1 << 26) + 1) == SHAPE and f(M=(1 << 26) + 1) == SHAPE
    assert f(M=1 << 20, N=1 << 17) == SHAPE
    assert f(xq=A + 8) == ALIGN and f(wq=C + 4) == ALIGN and f(y=E + 2) == ALIGN
    assert f(sx=B + 2) == ALIGN and f(sw=D + 1) == ALIGN
    assert f(y=A + 16) == ALIAS and f(y=C) == ALIAS and f(y=D) == ALIAS
    assert f(y=B - 4 * 130 * 2 + 16) == ALIAS  # its end reaches the scales
    assert f(M=0, xq=None, sx=None, y=None) == OK and f(N=0, wq=None, sw=None, y=None) == OK


def test_fp8_linear(lib):
    ws = lib.mq_fp8_linear_workspace_bytes
    assert ws(4, 272) == (4 * 272 + 255) // 256 * 256 + 4 * 3 * 4
    assert ws(0, 272) == 0 and ws(4, 270) == 0 and ws(-1, 272) == 0

    def f(x=A, wq=B, sw=C, y=D, M=4, N=130, K=272, w=E, n=None):
        return lib.mq_fp8_linear(x, wq, sw, y, M, N, K, w, ws(4, 272) if n is None else n, None)

    for k in ("x", "wq", "sw", "y"):
        assert f(**{k: None}) == NULL, k
    assert f(w=None) == WS and f(n=ws(4, 272) - 1) == WS
    assert f(w=E + 8) == ALIGN and f(w=A) == ALIAS and f(w=D + 16) == ALIAS and f(y=B) == ALIAS
    assert f(M=(1 << 26) + 1, K=16, N=1, n=1 << 40) == SHAPE and f(K=24) == SHAPE
    assert f(M=0, x=None, y=None, w=None, n=0) == OK


def test_wrappers_refuse_before_the_library():
    import torch
    x = torch.zeros((2, 32), dtype=torch.float16)
    with pytest.raises(ValueError):
        mq.rmsnorm_int8(x, torch.ones(32, dtype=torch.float16))  # not on a GPU
    with pytest.raises(TypeError):
        mq.quant_fp8_blocks(x.float())
    with pytest.raises(TypeError):
        mq.fp8_linear([1], None, None)
