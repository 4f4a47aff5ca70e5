"""RMS norm with 8-bit output of rows that hold a NaN or an infinity, or whose
residual sum leaves fp16's range: NaN scales, so that no product takes the row
for zeros; the other rows bit for bit."""

import numpy as np
import pytest

import weight_activation_quantized_amd as mq
import oracle
from oracle import fp8 as o8
from tests.fp8_util import codes_of, half_tensor
from tests.gpu_util import announce, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", ["fp16", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", [(7, 272), (7, 2048), (7, 4096), (200, 4096), (7, 8192), (130, 16384)])
def test_rows_that_are_not_finite(M, K, residual, half):
    rng = np.random.default_rng(K)
    x, w = rng.standard_normal((M, K)), 1 + 0.1 * rng.standard_normal(K)
    res = rng.standard_normal((M, K)) if residual else None
    big = 60000.0 if half == "fp16" else 3e38
    x[0, 3], x[2, K - 1], x[4, K // 2] = np.nan, np.inf, -np.inf
    lost = [0, 2, 4]
    if residual:
        x[5, 9] = res[5, 9] = big
        lost.append(5)
    (tx, xf), (tw, wf) = half_tensor(x, half), half_tensor(w, half)
    tr, rf = half_tensor(res, half) if residual else (None, None)
    keep = np.setdiff1d(np.arange(M), lost)
    v, _ = o8.rmsnorm_ref(xf[keep], wf, 1e-5, None if rf is None else rf[keep], half)
    announce(f"rmsnorm not finite {half} {M}x{K} residual={residual}")
    q, s = mq.rmsnorm_int8(tx, tw, 1e-5, residual=tr)[:2]
    s = host(s)
    want, ws = oracle.quant_per_token_int8_ref(v)
    assert np.isnan(s[lost]).all() and not host(q)[lost].any()
    assert np.array_equal(s[keep], ws) and np.array_equal(host(q)[keep], want)
    q, s = mq.rmsnorm_fp8(tx, tw, 1e-5, residual=tr)[:2]
    s = host(s)
    want, ws = o8.quant_fp8_blocks_ref(v)
    assert np.isnan(s[:, lost]).all() and not codes_of(q)[lost].any()
    assert np.array_equal(s[:, keep], ws) and np.array_equal(codes_of(q)[keep], want)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_their_layers_outputs(M):
    """The e4m3 and int8 products of such a row are NaN, the others finite."""
    import torch
    x = torch.randn((M, 512), dtype=torch.float16, device="cuda")
    x[1, 7] = float("inf")
    gain = torch.ones(512, dtype=torch.float16, device="cuda")
    announce(f"layers after a norm that is not finite, {M}")
    xq, s = mq.rmsnorm_fp8(x, gain)
    wq = torch.randn((256, 512), device="cuda").to(torch.float8_e4m3fn)
    y = mq.fp8_block_mm(xq, s, wq, torch.full((2, 4), 0.01, device="cuda"))
    xq, s = mq.rmsnorm_int8(x, gain)
    wi = torch.randint(-127, 128, (256, 512), dtype=torch.int8, device="cuda")
    z = mq.w8a8_scaled_mm(xq, s, wi, torch.full((256,), 0.01, device="cuda"))
    for out in (y, z):
        bad = host(torch.isnan(out))
        assert bad[1].all() and not np.delete(bad, 1, 0).any()
