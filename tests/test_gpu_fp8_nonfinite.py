"""NaN and infinities in the e4m3 linear layer's inputs: their rows' outputs are
NaN, in every form of the product, and no other row's change."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
from tests.fp8_util import half_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 300, 512), (16, 300, 4096), (40, 512, 12288), (100, 300, 400), (300, 1030, 2048),
                                   (1500, 2048, 1024)])
def test_linear(M, N, K, half):
    import torch
    rng = np.random.default_rng(M)
    wq = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda().to(torch.float8_e4m3fn)
    sw = torch.full((-(-N // 128), -(-K // 128)), 0.05, device="cuda")
    x, _ = half_tensor(rng.standard_normal((M, K)), half)
    announce(f"fp8_linear not finite {half} {M}x{K}x{N}")
    plain = host(mq.fp8_linear(x, wq, sw).float())
    rows = {0: float("nan"), 1: float("inf"), M - 1: float("-inf")}
    for m, bad in rows.items():
        x[m, int(rng.integers(0, K))] = bad
    got = host(mq.fp8_linear(x, wq, sw).float())
    staged = host(mq.fp8_block_mm(*mq.quant_fp8_blocks(x), wq, sw, out_dtype=x.dtype).float())
    assert np.isnan(got[list(rows)]).all() and np.isfinite(plain).all()
    assert np.array_equal(np.delete(got, list(rows), 0), np.delete(plain, list(rows), 0))
    assert np.array_equal(got, staged, equal_nan=True)
