"""Refusals of the drafted tokens' entry points on the CPU: bad arguments are
rejected on the host before any HIP call (the pointers are fake addresses)."""

import pytest

import weight_activation_quantized_amd as mq

OK, NULL, SHAPE, ALIGN, UNSUP, WS, ALIAS, HIP = range(8)
AT = {n: 0x10_0000_0000 * (i + 1) for i, n in enumerate(
    ["q", "k", "v", "qo", "cs", "pos", "qw", "kw", "kc", "vc", "ks", "vs", "table", "cu", "lens", "tree", "out", "ws",
     "parents", "probs", "draft", "tokens", "uniform", "kept", "path", "next"])}
SIZES = dict(T=10, B=3, Hq=8, Hkv=2, D=128, page=16, P=20, width=8, mq=4, rot=128, max_pos=100, words=1, layers=2)


@pytest.fixture(scope="module")
def lib():
    return mq.library()


def _args(kw):
    return {**AT, **SIZES, **kw}


def _cache(a):
    return [a[n] for n in ("kc", "vc", "ks", "vs", "table", "cu", "lens")]


def rope(lib, name="mq_kv8_rope_append", **kw):
    a = _args({"eps": 1e-6, "next": 0, "sq": None, "sk": None, "sv": None, "so": None, **kw})
    row, kv = a["Hq"] * a["D"], a["Hkv"] * a["D"]
    sq, so = (row if a[n] is None else a[n] for n in ("sq", "so"))
    sk, sv = (kv if a[n] is None else a[n] for n in ("sk", "sv"))
    return getattr(lib, name)(a["q"], a["k"], a["v"], sq, sk, sv, a["qo"], so, a["cs"], a["pos"], a["qw"], a["kw"],
                              a["eps"], a["max_pos"], a["rot"], a["next"], *_cache(a), a["T"], a["B"], a["Hq"], a["Hkv"],
                              a["D"], a["page"], a["P"], a["width"], a["mq"], None)


def attend(lib, **kw):
    a = _args({"scale": 0.1, "n": 1 << 40, **kw})
    return lib.mq_kv8_tree_attention(a["q"], a["Hq"] * a["D"], a["tree"], a["words"], *_cache(a), a["out"], a["T"], a["B"],
                                     a["Hq"], a["Hkv"], a["D"], a["page"], a["P"], a["width"], a["mq"], a["scale"], a["ws"],
                                     a["n"], None)


def keep(lib, **kw):
    a = _args({"nodes": 4, **kw})
    return lib.mq_kv8_tree_keep(*_cache(a), a["path"], a["kept"], a["layers"], a["B"], a["Hkv"], a["D"], a["page"], a["P"],
                                a["width"], a["nodes"], None)


def mask(lib, **kw):
    a = _args(kw)
    return lib.mq_kv8_tree_mask(a["parents"], a["cu"], a["lens"], a["tree"], a["pos"], a["T"], a["B"], a["words"], a["mq"],
                                None)


def verify(lib, **kw):
    a = _args({"draft": None, "V": 1000, "n": 1 << 40, **kw})
    return lib.mq_draft_verify(a["probs"], a["draft"], a["tokens"], a["parents"], a["uniform"], a["cu"], a["kept"],
                               a["path"], a["next"], a["T"], a["B"], a["V"], a["mq"], a["ws"], a["n"], None)


@pytest.mark.parametrize("call", [rope, attend, keep])
def test_cache_arguments(lib, call):
    for n in ("kc", "vc", "ks", "vs", "table", "cu", "lens"):
        assert call(lib, **{n: None}) == NULL, n
        assert call(lib, **{n: AT[n] + 2}) == ALIGN, n
    for D in (0, 32, 96, 256):
        assert call(lib, D=D) == UNSUP
    for page in (0, 8, 48, 256):
        assert call(lib, page=page) == UNSUP
    assert call(lib, B=-1) == SHAPE and call(lib, B=65536) == SHAPE
    assert call(lib, Hkv=0) == SHAPE and call(lib, Hkv=1025, Hq=1025) == SHAPE
    assert call(lib, P=0) == SHAPE and call(lib, width=0) == SHAPE and call(lib, width=(1 << 26) + 1) == SHAPE
    assert call(lib, B=0, table=None, cu=None, lens=None, kept=None, path=None) == OK


@pytest.mark.parametrize("name", ["mq_kv8_rope_append", "mq_kv8_rope_append_bf16"])
def test_rope_append(lib, name):
    def f(**kw):
        return rope(lib, name, **kw)

    for n in ("q", "k", "v", "qo", "cs"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: AT[n] + 8}) == ALIGN, n
    assert f(qw=None) == NULL and f(kw=None) == NULL  # together or not at all
    assert f(qw=AT["qw"] + 8) == ALIGN and f(kw=AT["kw"] + 2) == ALIGN and f(pos=AT["pos"] + 2) == ALIGN
    for rot in (0, 8, 24, 144, -16):
        assert f(rot=rot) == UNSUP
    assert f(D=64, rot=128) == UNSUP
    assert f(max_pos=0) == SHAPE and f(max_pos=(1 << 30) + 1) == SHAPE
    assert f(next=2) == UNSUP and f(eps=-1.0) == UNSUP and f(eps=float("nan")) == UNSUP and f(eps=2.0) == UNSUP
    assert f(Hq=7) == SHAPE and f(Hq=2048) == SHAPE and f(T=-1) == SHAPE and f(mq=0) == SHAPE
    for s, w in (("sq", 1024), ("so", 1024), ("sk", 256), ("sv", 256)):
        assert f(**{s: w - 8}) == SHAPE and f(**{s: w + 4}) == SHAPE and f(**{s: -w}) == SHAPE, s
    for n in ("q", "k", "v", "cs", "pos", "qw", "kc", "vs", "table", "lens"):
        at = AT[n] if n == "q" else AT[n] - 64
        assert f(qo=at + (16 if n == "q" else 0)) == ALIAS, n
    assert f(k=AT["kc"] + 64) == ALIAS and f(cs=AT["vc"]) == ALIAS and f(pos=AT["ks"]) == ALIAS and f(kw=AT["kc"]) == ALIAS
    assert f(B=65535, Hkv=128, Hq=128, D=64, rot=64, T=1 << 20, mq=1 << 20, width=1) == SHAPE
    assert f(T=0, q=None, k=None, v=None, qo=None) == OK and f(T=0, qw=None, kw=None, pos=None) == OK


def test_rope_append_in_place(lib):
    """q_out over q: the same stride; k and v may lie between q's rows, not in them."""
    row = (8 + 2 * 2) * 128
    q = AT["q"]
    fused = dict(q=q, qo=q, k=q + 8 * 128 * 2, v=q + 10 * 128 * 2, sq=row, sk=row, sv=row)
    assert rope(lib, **fused, so=row, B=0) == OK
    assert rope(lib, **fused, so=row + 8, B=0) == ALIAS
    assert rope(lib, **{**fused, "k": q + 7 * 128 * 2}, so=row, B=0) == ALIAS  # in the last query head
    assert rope(lib, **{**fused, "v": q + 11 * 128 * 2}, so=row, B=0) == ALIAS  # reaches the next row's q
    assert rope(lib, **{**fused, "sk": row + 8}, so=row, B=0) == ALIAS  # another stride wanders through them
    assert rope(lib, **{**fused, "k": q - 4 * 128 * 2}, so=row, B=0) == OK  # k in front of q
    assert rope(lib, q=q, qo=q, B=0) == OK  # dense, k and v elsewhere


def test_tree_attention(lib):
    for n in ("q", "out", "tree"):
        assert attend(lib, **{n: None}) == NULL, n
        assert attend(lib, **{n: AT[n] + 2}) == ALIGN, n
    assert attend(lib, words=0) == SHAPE and attend(lib, mq=33) == SHAPE and attend(lib, mq=33, words=2, T=0) == OK
    assert attend(lib, mq=1025, words=40) == SHAPE and attend(lib, mq=0) == SHAPE
    assert attend(lib, Hq=7) == SHAPE and attend(lib, scale=-1.0) == UNSUP and attend(lib, scale=float("nan")) == UNSUP
    assert attend(lib, out=AT["tree"]) == ALIAS and attend(lib, out=AT["q"] + 512) == ALIAS
    ws = lib.mq_kv8_tree_attention_workspace_bytes
    need = ws(1, 1, 8, 2, 128, 64, 1000, 1)
    long = dict(T=1, B=1, page=64, width=1000, mq=1)
    assert need > 0 and attend(lib, **long, ws=None) == WS and attend(lib, **long, n=need - 1) == WS
    assert attend(lib, **long, ws=AT["tree"]) == ALIAS and attend(lib, **long, ws=AT["ws"] + 8) == ALIGN
    assert ws(1, 1, 8, 2, 128, 64, 1000, 1025) == 0 and ws(1, 1, 8, 2, 96, 64, 1000, 1) == 0 and ws(0, 1, 8, 2, 128, 64, 9, 1) == 0


def test_tree_mask(lib):
    for n in ("parents", "cu", "lens", "tree", "pos"):
        assert mask(lib, **{n: None}) == NULL, n
        assert mask(lib, **{n: AT[n] + 1}) == ALIGN, n
    assert mask(lib, words=0) == SHAPE and mask(lib, mq=33) == SHAPE and mask(lib, mq=1025, words=64) == SHAPE
    assert mask(lib, T=-1) == SHAPE and mask(lib, B=65536) == SHAPE and mask(lib, mq=0) == SHAPE
    assert mask(lib, tree=AT["parents"]) == ALIAS and mask(lib, pos=AT["tree"] + 4) == ALIAS and mask(lib, pos=AT["lens"]) == ALIAS
    assert mask(lib, T=0, parents=None, tree=None, pos=None) == OK and mask(lib, B=0, cu=None, lens=None) == OK


def test_draft_verify(lib):
    for n in ("probs", "tokens", "uniform", "cu", "kept", "path", "next"):
        assert verify(lib, **{n: None}) == NULL, n
        assert verify(lib, **{n: AT[n] + 2}) == ALIGN, n
    assert verify(lib, draft=AT["draft"]) == UNSUP  # parents too
    assert verify(lib, draft=AT["draft"] + 1, parents=None) == ALIGN
    assert verify(lib, V=0) == SHAPE and verify(lib, V=(1 << 24) + 1) == SHAPE and verify(lib, mq=1025) == SHAPE
    assert verify(lib, T=-1) == SHAPE and verify(lib, B=-1) == SHAPE and verify(lib, mq=0) == SHAPE
    assert verify(lib, kept=AT["probs"] + 400) == ALIAS and verify(lib, path=AT["kept"]) == ALIAS
    assert verify(lib, next=AT["cu"]) == ALIAS and verify(lib, V=200000, ws=AT["path"]) == ALIAS
    need = lib.mq_draft_verify_workspace_bytes(3, 200000, 4)
    assert need > 0 and verify(lib, V=200000, n=need - 1) == WS and verify(lib, V=200000, ws=None) == WS
    assert verify(lib, V=200000, ws=AT["ws"] + 8) == ALIGN
    assert lib.mq_draft_verify_workspace_bytes(3, 1000, 4) == 0  # one kernel
    assert lib.mq_draft_verify_workspace_bytes(3, 0, 4) == 0 and lib.mq_draft_verify_workspace_bytes(-1, 10, 4) == 0
    assert verify(lib, B=0, cu=None, kept=None, path=None, next=None, ws=None) == OK


def test_tree_keep(lib):
    for n in ("path", "kept"):
        assert keep(lib, **{n: None}) == NULL and keep(lib, **{n: AT[n] + 2}) == ALIGN, n
    assert keep(lib, nodes=0) == SHAPE and keep(lib, nodes=1025) == SHAPE
    assert keep(lib, layers=-1) == SHAPE and keep(lib, layers=65536) == SHAPE and keep(lib, layers=0) == OK
    assert keep(lib, path=AT["kc"] + 2 * 20 * 2 * 16 * 128 - 16) == ALIAS  # in the second layer
    assert keep(lib, kept=AT["vs"]) == ALIAS and keep(lib, kc=AT["vc"] + 64) == ALIAS
    assert keep(lib, B=65535, Hkv=1000) == SHAPE


def test_wrappers_refuse_before_the_library():
    import torch
    x, i = torch.zeros((2, 1, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mq.kv8_tree_mask(i, i, i, 2)  # not on a GPU
    with pytest.raises(TypeError):
        mq.kv8_tree_mask([0], i, i, 2)
    with pytest.raises(TypeError):
        mq.kv8_rope_append(x.float(), x, x, *[i] * 7, 1, x)
    with pytest.raises(ValueError):
        mq.draft_verify(torch.zeros(2, 5), i, torch.zeros(2), i, 2)
    with pytest.raises(ValueError):
        mq.kv8_tree_attention(x, i.view(2, 1), *[i] * 7, 1)
    with pytest.raises(ValueError):
        mq.kv8_tree_keep(*[i] * 9)


STREAMED = {
    "kv8_rope_append": lambda x, s: mq.kv8_rope_append(*[x] * 10, 1, x, stream=s),
    "kv8_tree_mask": lambda x, s: mq.kv8_tree_mask(x, x, x, 1, stream=s),
    "kv8_tree_attention": lambda x, s: mq.kv8_tree_attention(*[x] * 9, 1, stream=s),
    "draft_verify": lambda x, s: mq.draft_verify(x, x, x, x, 1, stream=s),
    "kv8_tree_keep": lambda x, s: mq.kv8_tree_keep(*[x] * 9, stream=s),
}


@pytest.mark.parametrize("name", STREAMED)
def test_stream_of_another_gpu(name, monkeypatch):
    import contextlib
    from types import SimpleNamespace

    import torch
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(mq, "_native_module", SimpleNamespace(**{name: lambda *a: "called"}))
    x = SimpleNamespace(device=torch.device("cuda", 0))
    one, other = (SimpleNamespace(device=torch.device("cuda", i)) for i in (0, 1))
    assert STREAMED[name](x, one) == "called"
    with pytest.raises(ValueError, match="stream of cuda:1 for tensors on cuda:0"):
        STREAMED[name](x, other)
