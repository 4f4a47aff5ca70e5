"""Outputs that the wrappers allocate are those of ``torch.empty``: filled under
``torch.use_deterministic_algorithms``, seen by dispatch modes."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from tests.draft_util import offsets, words_of
from tests.fp8_util import codes_tensor, half_tensor
from tests.gpu_util import announce, host
from tests.kv8_util import paged, up

pytestmark = pytest.mark.gpu

NEWS, TOTALS, PAD = [4, 3], [40, 9], 5


def _calls():
    """Name -> a call whose last PAD rows are rows of no sequence."""
    rng = np.random.default_rng(0)
    cache, table = paged(rng, TOTALS, 2, 16, 64)
    cu, T = offsets(NEWS), sum(NEWS) + PAD
    dev = codes_tensor(cache[0]), codes_tensor(cache[1]), up(cache[2]), up(cache[3])
    batch = up(table), up(cu), up(np.array(TOTALS, np.int32))
    q, _ = half_tensor(rng.standard_normal((T, 4, 64)), "fp16")
    k, _ = half_tensor(rng.standard_normal((T, 2, 64)), "fp16")
    parents = np.concatenate([np.arange(-1, n - 1) for n in NEWS] + [np.zeros(PAD)]).astype(np.int32)
    tree = up(np.concatenate([words_of(parents[:-PAD], NEWS, TOTALS), np.zeros((PAD, 1), np.int32)]))
    angles = up(rng.standard_normal((64, 32)).astype(np.float32))
    return {
        "kv8_attention": lambda: mq.kv8_attention(q, *dev, *batch, 4),
        "kv8_tree_attention": lambda: mq.kv8_tree_attention(q, tree, *dev, *batch, 4),
        "kv8_rope_append": lambda: mq.kv8_rope_append(q, k, k, *dev, *batch, 4, angles),
        "kv8_tree_mask": lambda: mq.kv8_tree_mask(up(parents), *batch[1:], 4),
    }


@pytest.mark.parametrize("name", ["kv8_attention", "kv8_tree_attention", "kv8_rope_append", "kv8_tree_mask"])
def test_filled_where_torch_fills(name):
    import torch
    call = _calls()[name]
    junk = [torch.zeros(1 << n, dtype=torch.uint8, device="cuda") for n in range(6, 16) for _ in range(8)]
    del junk  # (what the allocator hands out next holds zeros)
    torch.use_deterministic_algorithms(True)
    try:
        announce(f"{name}, deterministic")
        got = call()
    finally:
        torch.use_deterministic_algorithms(False)
    for t in got if isinstance(got, tuple) else (got,):
        rest = host(t[sum(NEWS):].float() if t.is_floating_point() else t[sum(NEWS):])
        assert np.all(np.isnan(rest)) if t.is_floating_point() else np.all(rest == 2 ** 31 - 1)


@pytest.mark.parametrize("name", ["kv8_attention", "kv8_tree_attention", "kv8_rope_append", "kv8_tree_mask"])
def test_seen_by_dispatch_modes(name):
    import torch
    from torch.utils._python_dispatch import TorchDispatchMode
    seen = []

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(func)
            return func(*args, **(kwargs or {}))

    call = _calls()[name]
    announce(f"{name}, watched")
    with Watch():
        got = call()
    assert seen.count(torch.ops.aten.empty.memory_format) >= (2 if isinstance(got, tuple) else 1)
