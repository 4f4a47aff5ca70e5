// RMS norm with the residual's addition and 8-bit output, and the e4m3
// quantizer per 128 values, for gfx950.
//
//   h = rne16(x + residual)            (or x; x, residual, w fp16 or bf16)
//   r = fl32(1 / sqrt(sum_k h^2 / K + eps))    in binary64
//   v = fl32(fl32(h * r) * w)
//   int8: s = fl32(max|v| / 127) per row,         q = clamp(rne(fl32(v / s)), -127, 127)
//   e4m3: s = fl32(max|v| / 448) per 128 values,  q = rne_e4m3(clamp(fl32(v / s), -448, 448))
//
// The squares are added in binary64 (each square of a 16-bit value is exact
// there), so r, and with it every code and scale, does not depend on the
// order of the sum: a last bit of r would move codes that sit next to a
// rounding border. It costs two 64-bit VALU operations per value of a kernel
// bound by HBM.
//
// A row stays in registers (16-byte chunks of 8 values), so x and residual
// are read once and h and the codes written once: 7 bytes per value with a
// residual, 3 without. The 128 values that share an e4m3 scale are 16
// consecutive chunks, one row of 16 lanes, so their maximum takes four DPP
// steps and no LDS. The scales go out transposed, [K / 128, M]: the product
// that reads them wants the scales of neighbouring tokens side by side.
//
// 8192 rows of 4096 with a residual: 47 us captured, 45 called eagerly one after
// the other, 5.2 TB/s, the kernel alone 39.5 in a trace. Small calls are a launch
// and two passes of latency, captured one row of 4096 3.1 us, 333 of 5008 4.5.
// The quantizer alone, captured: 517 rows of 4096 4.0 us, 4096 14.1, 32768 94.7,
// 4.3 TB/s.
#include "block8_launch.h"
#include "device_common.h"
#include "quant_codes.h"

namespace mq {
namespace {

template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double x) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  const int lo = static_cast<int>(b[0]), hi = static_cast<int>(b[1]);
  return __builtin_bit_cast(double, u32x2{static_cast<uint32_t>(__builtin_amdgcn_update_dpp(lo, lo, kCtrl, 0xF, 0xF, false)),
                                          static_cast<uint32_t>(__builtin_amdgcn_update_dpp(hi, hi, kCtrl, 0xF, 0xF, false))});
}

__device__ __forceinline__ double lane_f64(double x, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  return __builtin_bit_cast(double, u32x2{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b[0]), lane)),
                                          static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b[1]), lane))});
}

// Sum over the wavefront, the same value in every lane.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_f64<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp_f64<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp_f64<0x141>(v);  // row_half_mirror
  v += dpp_f64<0x140>(v);  // row_mirror: every lane holds its row's sum
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// kTh threads per row (64: four rows per workgroup of 256; otherwise one row
// per workgroup), CPT 16-byte chunks per thread: K <= 8 kTh CPT.
template <int kTh, int CPT, bool kFp8, bool kBf16, bool kRes>
__global__ __launch_bounds__(kTh == 64 ? 256 : kTh) void rmsnorm_quant_kernel(
    const uint16_t* __restrict__ x, const uint16_t* residual, const uint16_t* __restrict__ weight, double eps,
    uint16_t* h_out, uint8_t* __restrict__ codes, float* __restrict__ scales, int M, int K) {
  constexpr int kWaves = kTh / 64;
  __shared__ double wsum[kWaves];
  __shared__ float wmax[kWaves];
  const int t = kTh == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int row = kTh == 64 ? static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 6)
                            : static_cast<int>(blockIdx.x);
  if (kTh == 64 && row >= M) return;  // whole wavefronts; no barrier follows in this form
  const int nchunk = K >> 3;
  const size_t base = static_cast<size_t>(row) * K;

  u32x4 v[CPT], rs[CPT], wt[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + kTh * i;
    v[i] = rs[i] = wt[i] = u32x4{0u, 0u, 0u, 0u};
    if (c < nchunk) {
      v[i] = *reinterpret_cast<const u32x4*>(x + base + 8 * c);
      if constexpr (kRes) rs[i] = *reinterpret_cast<const u32x4*>(residual + base + 8 * c);
      wt[i] = *reinterpret_cast<const u32x4*>(weight + 8 * c);
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float lo, hi;
      word_to_floats<kBf16>(v[i][w], lo, hi);
      if constexpr (kRes) {
        float a, b;
        word_to_floats<kBf16>(rs[i][w], a, b);
        v[i][w] = static_cast<uint32_t>(half_bits<kBf16>(lo + a)) |
                  (static_cast<uint32_t>(half_bits<kBf16>(hi + b)) << 16);
        word_to_floats<kBf16>(v[i][w], lo, hi);
      }
      sum = fma(static_cast<double>(lo), static_cast<double>(lo), sum);
      sum = fma(static_cast<double>(hi), static_cast<double>(hi), sum);
    }
    if constexpr (kRes) {
      const int c = t + kTh * i;
      if (c < nchunk) *reinterpret_cast<u32x4*>(h_out + base + 8 * c) = v[i];
    }
  }
  sum = wave_sum(sum);
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = wsum[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += wsum[w];
  }
  const float r = static_cast<float>(1.0 / sqrt(sum / static_cast<double>(K) + eps));
  // A NaN or infinity in the row (a residual sum past fp16's range, say): maxima
  // skip NaN and the codes have none, so the scales say it.
  const bool lost = !(sum < static_cast<double>(__builtin_inff()));

  float f[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float lo, hi, a, b;
      word_to_floats<kBf16>(v[i][w], lo, hi);
      word_to_floats<kBf16>(wt[i][w], a, b);
      f[i][2 * w] = (lo * r) * a;
      f[i][2 * w + 1] = (hi * r) * b;
    }
  }
  if constexpr (kFp8) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[i][e]));
      const float s = lost ? __builtin_nanf("") : row16_max(m) / kE4m3Max;
      const int c = t + kTh * i;
      if (c >= nchunk) continue;
      *reinterpret_cast<u32x2*>(codes + base + 8 * c) = e4m3_codes(f[i], s, __builtin_amdgcn_rcpf(s));
      if ((c & 15) == 0) scales[static_cast<size_t>(c >> 4) * M + row] = s;
    }
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[i][e]));
    m = wave_max(m);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
      __syncthreads();
      m = wmax[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) m = fmaxf(m, wmax[w]);
    }
    const float s = lost ? __builtin_nanf("") : m / 127.0f;
    const float rc = code_rcp(s);
    if (t == 0) scales[row] = s;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + kTh * i;
      if (c < nchunk) *reinterpret_cast<u32x2*>(codes + base + 8 * c) = int8_codes(f[i], s, rc);
    }
  }
}

// e4m3 codes and scales of x: 16 lanes take one block of 128 values, so a
// wavefront covers 4 blocks and every block is on its own. The grid's y walks
// the row in steps of 256 chunks.
template <bool kBf16>
__global__ __launch_bounds__(256) void quant_fp8_blocks_kernel(const uint16_t* __restrict__ x,
                                                               uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales, int64_t M, int nchunk,
                                                               int wide) {
  // `wide` 16-lane groups per row; consecutive groups take consecutive blocks
  // (fewer than 2^31 groups: the 2^38 values behind them fit no memory)
  const uint32_t g = blockIdx.x * 16 + (threadIdx.x >> 4);
  const uint32_t row = g / static_cast<uint32_t>(wide);
  const int c = static_cast<int>(g - row * wide) * 16 + static_cast<int>(threadIdx.x & 15);
  const bool in = row < M && c < nchunk;
  u32x4 v = {0u, 0u, 0u, 0u};
  const size_t at = (static_cast<size_t>(row) * nchunk + c) * 8;
  if (in) v = *reinterpret_cast<const u32x4*>(x + at);
  float f[8], m = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    word_to_floats<kBf16>(v[w], f[2 * w], f[2 * w + 1]);
    m = fmaxf(m, fmaxf(fabsf(f[2 * w]), fabsf(f[2 * w + 1])));
  }
  const float s = row16_max(m) / kE4m3Max;
  if (!in) return;
  *reinterpret_cast<u32x2*>(codes + at) = e4m3_codes(f, s, __builtin_amdgcn_rcpf(s));
  if ((c & 15) == 0) scales[static_cast<size_t>(c >> 4) * M + row] = s;
}

template <int kTh, int CPT, bool kFp8, bool kBf16>
hipError_t launch_form(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps, uint16_t* h,
                       uint8_t* codes, float* scales, int M, int K, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(kTh == 64 ? (M + 3) / 4 : M)), block(kTh == 64 ? 256 : kTh);
  if (residual != nullptr)
    return launch_kernel(rmsnorm_quant_kernel<kTh, CPT, kFp8, kBf16, true>, grid, block, 0, stream, x, residual, weight,
                         eps, h, codes, scales, M, K);
  return launch_kernel(rmsnorm_quant_kernel<kTh, CPT, kFp8, kBf16, false>, grid, block, 0, stream, x, residual, weight,
                       eps, h, codes, scales, M, K);
}

template <bool kFp8, bool kBf16>
hipError_t launch_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps, uint16_t* h,
                       uint8_t* codes, float* scales, int M, int K, hipStream_t stream) {
  const int chunks = K / 8;
#define MQ_FORM(TH, C) return launch_form<TH, C, kFp8, kBf16>(x, residual, weight, eps, h, codes, scales, M, K, stream)
  if (chunks <= 64) MQ_FORM(64, 1);
  if (chunks <= 256) MQ_FORM(256, 1);
  // few rows: a chunk per thread (one row of 4096 captured: 3.1 us, with 256 threads 3.2)
  if (M <= 128 && chunks <= 512) MQ_FORM(512, 1);
  if (M <= 128 && chunks <= 1024) MQ_FORM(1024, 1);
  if (chunks <= 512) MQ_FORM(256, 2);
  if (chunks <= 1024) MQ_FORM(256, 4);
  if (chunks <= 2048) MQ_FORM(1024, 2);
  if (chunks <= 4096) MQ_FORM(1024, 4);
  MQ_FORM(1024, 8);
#undef MQ_FORM
}

}  // namespace

hipError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps,
                                uint16_t* h, uint8_t* codes, float* scales, int64_t M, int64_t K, bool fp8, bool bf16,
                                hipStream_t stream) {
  if (K > kRmsnormMaxK) return hipErrorInvalidValue;
  const int m = static_cast<int>(M), k = static_cast<int>(K);
  if (fp8)
    return bf16 ? launch_norm<true, true>(x, residual, weight, eps, h, codes, scales, m, k, stream)
                : launch_norm<true, false>(x, residual, weight, eps, h, codes, scales, m, k, stream);
  return bf16 ? launch_norm<false, true>(x, residual, weight, eps, h, codes, scales, m, k, stream)
              : launch_norm<false, false>(x, residual, weight, eps, h, codes, scales, m, k, stream);
}

hipError_t launch_quant_fp8_blocks(const uint16_t* x, uint8_t* codes, float* scales, int64_t M, int64_t K, bool bf16,
                                   hipStream_t stream) {
  const int nchunk = static_cast<int>(K / 8), wide = (nchunk + 15) / 16;
  const int64_t blocks = (M * wide + 15) / 16;
  if (blocks >= (int64_t{1} << 27)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(blocks)), block(256);
  return bf16 ? launch_kernel(quant_fp8_blocks_kernel<true>, grid, block, 0, stream, x, codes, scales, M, nchunk, wide)
              : launch_kernel(quant_fp8_blocks_kernel<false>, grid, block, 0, stream, x, codes, scales, M, nchunk, wide);
}

}  // namespace mq
