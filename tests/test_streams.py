"""The ``stream`` argument of the wrappers with a native half, on the CPU: a
stream of another GPU than the tensors' is refused."""

from types import SimpleNamespace

import pytest

import weight_activation_quantized_amd as mq

CALLS = {
    "rmsnorm_int8": lambda x, s: mq.rmsnorm_int8(x, x, stream=s),
    "rmsnorm_fp8": lambda x, s: mq.rmsnorm_fp8(x, x, stream=s),
    "quant_fp8_blocks": lambda x, s: mq.quant_fp8_blocks(x, stream=s),
    "fp8_block_mm": lambda x, s: mq.fp8_block_mm(x, x, x, x, stream=s),
    "fp8_linear": lambda x, s: mq.fp8_linear(x, x, x, stream=s),
    "kv8_append": lambda x, s: mq.kv8_append(x, x, x, x, x, x, x, x, x, 1, stream=s),
    "kv8_attention": lambda x, s: mq.kv8_attention(x, x, x, x, x, x, x, x, 1, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_gpu(name, monkeypatch):
    import torch
    ran = []

    class Current:
        def __init__(self, stream):
            ran.append(stream)

        def __enter__(self):
            pass

        def __exit__(self, *a):
            pass

    monkeypatch.setattr(torch.cuda, "stream", Current)
    native = SimpleNamespace(**{n: lambda *a: "called" for n in (
        "rmsnorm", "quant_fp8_blocks", "fp8_block_mm", "fp8_linear", "kv8_append", "kv8_attention")})
    monkeypatch.setattr(mq, "_native_module", native)
    x = SimpleNamespace(device=torch.device("cuda", 0))
    one, other = (SimpleNamespace(device=torch.device("cuda", i)) for i in (0, 1))
    assert CALLS[name](x, one) == "called" and ran == [one]
    with pytest.raises(ValueError, match="stream of cuda:1 for tensors on cuda:0"):
        CALLS[name](x, other)
    assert ran == [one]
