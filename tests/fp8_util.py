"""Helpers of the e4m3 operators' tests: 16-bit inputs of either format, e4m3
tensors from codes, and codes back."""

import numpy as np

import synth


def half_tensor(values, half, device="cuda"):
    """float32 values -> (torch tensor of the format, the values it holds)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32))
    t = t.to(torch.bfloat16 if half == "bf16" else torch.float16)
    return t.to(device), t.float().numpy()


def codes_tensor(codes, device="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(codes)).to(device).view(torch.float8_e4m3fn)


def codes_of(t):
    import torch
    torch.cuda.synchronize()
    return t.view(torch.uint8).cpu().numpy()


def random_codes(rng, shape):
    """Finite e4m3 codes, every one of them equally likely."""
    c = rng.integers(0, 254, size=shape, dtype=np.uint8)
    return np.where(c >= 127, c + 1, c).astype(np.uint8)  # skips 0x7F; 0xFF is never drawn


def activations(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    cols = rng.choice(K, size=max(1, K // 100), replace=False)
    x[:, cols] *= synth.OUTLIER_GAIN
    return x


def group_max_sum(xq, s_x, wq, s_w):
    """sum over groups of 8 consecutive k of the largest |x w| in the group, for
    every (m, n): the scale of what the fp8 matrix unit drops. Plain products
    and maxima in float64 on the GPU, a few channels at a time."""
    import torch
    from oracle import fp8 as o8
    M, K = xq.shape
    N = wq.shape[0]
    kb, nb = np.arange(K) // 128, np.arange(N) // 128
    x = torch.from_numpy(np.abs(o8.e4m3_decode(xq) * s_x.astype(np.float64).T[:, kb])).cuda()
    w = torch.from_numpy(np.abs(o8.e4m3_decode(wq) * s_w.astype(np.float64)[nb][:, kb])).cuda()
    out = torch.empty((M, N), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // (M * K))
    for n in range(0, N, step):
        p = x[:, None, :] * w[None, n:n + step, :]
        out[:, n:n + step] = p.view(M, p.shape[1], K // 8, 8).amax(-1).sum(-1)
    return out.cpu().numpy()
