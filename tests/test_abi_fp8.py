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
    ws = lib.mq_fp8_block_mm_workspace_bytes

    def f(xq=A, sx=B, wq=C, sw=D, y=E, M=4, N=130, K=272, w=F, n=1 << 40):
        return lib.mq_fp8_block_mm(xq, sx, wq, sw, y, M, N, K, w, n, None)

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
    # few tiles and a long K are split, which needs a workspace
    long = dict(M=40, N=512, K=12288)
    need = ws(40, 512, 12288)
    assert need > 0 and need % (40 * 512 * 4) == 0
    assert f(**long, w=None) == WS and f(**long, n=need - 1) == WS and f(**long, w=F + 8) == ALIGN
    assert f(**long, w=A) == ALIAS and f(**long, w=E + 16) == ALIAS
    assert ws(4, 130, 272) == 0 and ws(-1, 512, 12288) == 0 and ws(40, 512, 12280) == 0 and ws(0, 512, 12288) == 0


def test_fp8_linear(lib):
    ws = lib.mq_fp8_linear_workspace_bytes
    assert ws(4, 130, 272) == 0  # one kernel
    need = ws(100, 130, 272)
    assert need >= 100 * 272 + 100 * 3 * 4
    assert ws(0, 130, 272) == 0 and ws(100, 130, 270) == 0 and ws(-1, 130, 272) == 0

    def f(x=A, wq=B, sw=C, y=D, M=100, N=130, K=272, w=E, n=None):
        return lib.mq_fp8_linear(x, wq, sw, y, M, N, K, w, need if n is None else n, None)

    for k in ("x", "wq", "sw", "y"):
        assert f(**{k: None}) == NULL, k
    assert f(w=None) == WS and f(n=need - 1) == WS
    assert f(w=E + 8) == ALIGN and f(w=A) == ALIAS and f(w=D + 16) == ALIAS and f(y=B) == ALIAS
    assert f(M=(1 << 26) + 1, K=16, N=1, n=1 << 40) == SHAPE and f(K=24) == SHAPE
    assert f(M=0, x=None, y=None, w=None, n=0) == OK
    assert f(M=4, y=C, n=0, w=None) == ALIAS


def test_wrappers_refuse_before_the_library():
    import torch
    x = torch.zeros((2, 32), dtype=torch.float16)
    with pytest.raises(ValueError):
        mq.rmsnorm_int8(x, torch.ones(32, dtype=torch.float16))  # not on a GPU
    with pytest.raises(TypeError):
        mq.quant_fp8_blocks(x.float())
    with pytest.raises(TypeError):
        mq.fp8_linear([1], None, None)


class Cache:
    """Arguments of the cache entry points with fake, far-apart addresses."""
    sizes = dict(T=10, B=3, Hkv=2, D=128, page=16, P=20, width=8, mq=4)
    at = {n: 0x10_0000_0000 * (i + 20) for i, n in enumerate(
        ["k", "v", "q", "kc", "vc", "ks", "vs", "table", "cu", "lens", "out", "ws"])}


def _append(lib, **kw):
    a = {**Cache.sizes, **Cache.at, "sk": None, "sv": None, **kw}
    sk = a["Hkv"] * a["D"] if a["sk"] is None else a["sk"]
    sv = a["Hkv"] * a["D"] if a["sv"] is None else a["sv"]
    return lib.mq_kv8_append(a["k"], a["v"], sk, sv, a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["cu"], a["lens"],
                             a["T"], a["B"], a["Hkv"], a["D"], a["page"], a["P"], a["width"], a["mq"], None)


def _attention(lib, **kw):
    a = {**Cache.sizes, **Cache.at, "sq": None, "Hq": 8, "scale": 0.1, "n": 1 << 40, **kw}
    sq = a["Hq"] * a["D"] if a["sq"] is None else a["sq"]
    return lib.mq_kv8_attention(a["q"], sq, a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["cu"], a["lens"], a["out"],
                                a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], a["page"], a["P"], a["width"], a["mq"],
                                a["scale"], a["ws"], a["n"], None)


@pytest.mark.parametrize("call", [_append, _attention])
def test_kv8_cache_arguments(lib, call):
    for n in ("kc", "vc", "ks", "vs", "table", "cu", "lens"):
        assert call(lib, **{n: None}) == NULL, n
    for D in (0, 32, 96, 256):
        assert call(lib, D=D) == UNSUP
    for page in (0, 8, 48, 256):
        assert call(lib, page=page) == UNSUP
    assert call(lib, T=-1) == SHAPE and call(lib, T=(1 << 26) + 1) == SHAPE
    assert call(lib, B=-1) == SHAPE and call(lib, B=65536) == SHAPE
    assert call(lib, Hkv=0) == SHAPE and call(lib, Hkv=1025) == SHAPE
    assert call(lib, P=0) == SHAPE and call(lib, width=0) == SHAPE and call(lib, width=(1 << 26) + 1) == SHAPE
    assert call(lib, mq=0) == SHAPE
    assert call(lib, kc=Cache.at["kc"] + 8) == ALIGN and call(lib, vc=Cache.at["vc"] + 1) == ALIGN
    for n in ("ks", "vs", "table", "cu", "lens"):
        assert call(lib, **{n: Cache.at[n] + 2}) == ALIGN, n
    assert call(lib, T=0, k=None, v=None, q=None, out=None) == OK and call(lib, B=0, table=None, cu=None, lens=None) == OK


def test_kv8_append_arguments(lib):
    assert _append(lib, k=None) == NULL and _append(lib, v=None) == NULL
    assert _append(lib, sk=255) == SHAPE and _append(lib, sv=260) == SHAPE and _append(lib, sk=-256) == SHAPE
    assert _append(lib, k=Cache.at["k"] + 8) == ALIGN and _append(lib, v=Cache.at["v"] + 2) == ALIGN
    assert _append(lib, k=Cache.at["kc"] + 64) == ALIAS and _append(lib, vc=Cache.at["kc"] + 1024) == ALIAS
    assert _append(lib, ks=Cache.at["vs"] + 4) == ALIAS and _append(lib, lens=Cache.at["ks"]) == ALIAS
    # the last row's end reaches the cache through the stride alone
    assert _append(lib, k=Cache.at["kc"] - 10 * 256 * 2, sk=512) == ALIAS
    assert _append(lib, B=65535, Hkv=128, D=64, T=1 << 20, mq=1 << 20, width=1) == SHAPE


def test_kv8_attention_arguments(lib):
    ws = lib.mq_kv8_attention_workspace_bytes
    assert _attention(lib, q=None) == NULL and _attention(lib, out=None) == NULL
    assert _attention(lib, Hq=7) == SHAPE and _attention(lib, Hq=0) == SHAPE and _attention(lib, Hq=2048) == SHAPE
    assert _attention(lib, sq=1000) == SHAPE and _attention(lib, q=Cache.at["q"] + 4) == ALIGN
    assert _attention(lib, scale=float("nan")) == UNSUP and _attention(lib, scale=float("inf")) == UNSUP
    assert _attention(lib, scale=-0.1) == UNSUP and _attention(lib, T=0, q=None, out=None, scale=0.0) == OK
    assert _attention(lib, out=Cache.at["q"] + 512) == ALIAS and _attention(lib, out=Cache.at["kc"]) == ALIAS
    assert _attention(lib, out=Cache.at["out"] + 8) == ALIGN
    # a long sequence needs a workspace
    need = ws(1, 1, 8, 2, 128, 64, 1000, 1)
    assert need > 0
    long = dict(T=1, B=1, page=64, width=1000, mq=1)
    assert _attention(lib, **long, ws=None) == WS and _attention(lib, **long, n=need - 1) == WS
    assert _attention(lib, **long, ws=Cache.at["ws"] + 8) == ALIGN and _attention(lib, **long, ws=Cache.at["kc"]) == ALIAS
    assert _attention(lib, **long, ws=Cache.at["out"]) == ALIAS
    assert ws(1, 1, 7, 2, 128, 64, 1000, 1) == 0 and ws(1, 1, 8, 2, 96, 64, 1000, 1) == 0 and ws(0, 1, 8, 2, 128, 64, 9, 1) == 0
