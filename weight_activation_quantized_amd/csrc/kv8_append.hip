// Append to the paged e4m3 KV cache, for gfx950.
//
// One scale serves the tokens of one page and kv head (K and V apart). With a
// the largest |x| among the new tokens that fall into the page,
//   s_new = 2^ceil(log2(a / 448)), its exponent held in [-100, 120]
//   s     = s_new                      where the page held no older token
//         = max(s_old, s_new)          otherwise
// new codes are rne_e4m3(x / s), and where s grew, older codes become
// rne_e4m3(code * s_old / s). Powers of two: a 4-bit significand loses nothing
// to a scale up to twice too large, and moving older codes to a larger scale
// only shifts their exponents (codes that fall below 2^-6 round, nothing else).
//
// A workgroup owns one (sequence, page, head, K or V): the new rows of the
// page stay in registers between the maximum and the codes, so they are read
// once, and nothing is shared between workgroups (no atomics, the same bits
// every time). K rows go out as they come. V pages are stored transposed,
// [head_dim, page]: the attention's second product then reads 16 tokens of one
// dimension with one load; the transposition happens here, once per token, in
// LDS.
#include "device_common.h"
#include "launch.h"
#include "quant_codes.h"

namespace mq {
namespace {

constexpr int kThreads = 256;

// Smallest power of two s with a <= 448 s, its exponent held in [-100, 120].
// 448 = 1.75 * 2^8: with a = 1.m * 2^e the exponent is e - 8 for a fraction up
// to .75 and e - 7 above, which the carry out of the fraction adds.
__device__ __forceinline__ float page_scale(float a) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, a) & 0x7fffffffu;
  int e = static_cast<int>((bits + 0x1fffffu) >> 23) - 127 - 8;
  e = min(max(e, -100), 120);
  return __builtin_bit_cast(float, static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float clamp448(float v) { return __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max); }

// The four codes of a word times ratio, rounded to e4m3 again.
__device__ __forceinline__ uint32_t moved(uint32_t w, float ratio) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  return e4m3x4(clamp448(a[0] * ratio), clamp448(a[1] * ratio), clamp448(b[0] * ratio), clamp448(b[1] * ratio));
}

// CPT: 16-byte chunks (8 values) of a page's rows per thread.
template <int D, int CPT, bool kBf16>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Cache c, const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, int64_t k_stride,
                                                              int64_t v_stride, int span) {
  constexpr int kDc = D / 8;  // chunks per row
  __shared__ float wmax[kThreads / 64];
  __shared__ __attribute__((aligned(16))) uint8_t tile[D * (128 + 16)];

  // blockIdx.x = ((sequence * span + page) * kv_heads + head) * 2 + (0: K, 1: V)
  unsigned at = blockIdx.x;
  const bool is_v = at & 1;
  at >>= 1;
  const int head = static_cast<int>(at % c.kv_heads);
  at /= c.kv_heads;
  const int b = static_cast<int>(at / span);
  const int first_row = c.cu[b], n = c.cu[b + 1] - first_row, len = c.lens[b];
  if (n <= 0 || len <= 0) return;
  const int start = len - n;  // position of the first new token
  const int slot = (max(start, 0) >> c.page_shift) + static_cast<int>(at % span);
  if (slot >= c.table_width) return;
  const int64_t pos0 = static_cast<int64_t>(slot) * c.page;
  if (pos0 >= len) return;
  const int id = c.table[static_cast<size_t>(b) * c.table_width + slot];
  if (id < 0 || id >= c.num_pages) return;
  const int lo = max(start - static_cast<int>(pos0), 0);                    // first new token of the page
  // behind the last (a sequence longer than max_q_len is cut to what the
  // registers hold, never read or written past them)
  const int hi = min(min(len - static_cast<int>(pos0), c.page), lo + CPT * kThreads / kDc);
  const int64_t row0 = first_row + pos0 - start;  // row of the page's token 0

  const uint16_t* const x = is_v ? v : k;
  const int64_t stride = is_v ? v_stride : k_stride;
  u32x4 w[CPT];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int ch = static_cast<int>(threadIdx.x) + kThreads * i;
    const int t = lo + ch / kDc;
    const int64_t row = row0 + t;
    w[i] = u32x4{0u, 0u, 0u, 0u};
    if (t < hi && row >= 0 && row < c.tokens)
      w[i] = *reinterpret_cast<const u32x4*>(x + row * stride + head * D + 8 * (ch % kDc));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, z;
      word_to_floats<kBf16>(w[i][e], a, z);
      amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(z)));
    }
  }
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));

  const size_t unit = static_cast<size_t>(id) * c.kv_heads + head;
  float* const scale_at = (is_v ? c.v_scales : c.k_scales) + unit;
  uint8_t* const out = (is_v ? c.v : c.k) + unit * c.page * D;
  float s = page_scale(amax);
  if (lo > 0) {  // the page holds older tokens
    const float old = *scale_at;
    if (s > old) {
      const float ratio = old / s;
      if (!is_v) {
        for (int i = threadIdx.x; i < lo * D / 4; i += kThreads) {
          uint32_t* const p = reinterpret_cast<uint32_t*>(out) + i;
          *p = moved(*p, ratio);
        }
      } else {
        // words of four tokens of one dimension; the tokens from lo on keep
        // their bytes (new ones are written after the barrier)
        const int words = (lo + 3) / 4;
        for (int i = threadIdx.x; i < words * D; i += kThreads) {
          const int d = i / words, wd = i - d * words;
          uint32_t* const p = reinterpret_cast<uint32_t*>(out + static_cast<size_t>(d) * c.page + 4 * wd);
          const int keep = min(lo - 4 * wd, 4);
          const uint32_t mask = keep == 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
          const uint32_t before = *p;
          *p = (moved(before, ratio) & mask) | (before & ~mask);
        }
      }
    } else {
      s = old;
    }
  }
  __syncthreads();  // every lane has read the old scale, and older codes are in place
  if (threadIdx.x == 0) *scale_at = s;

#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int ch = static_cast<int>(threadIdx.x) + kThreads * i;
    const int t = lo + ch / kDc, d = 8 * (ch % kDc);
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, z;
      word_to_floats<kBf16>(w[i][e], a, z);
      f[2 * e] = clamp448(a / s);
      f[2 * e + 1] = clamp448(z / s);
    }
    const u32x2 codes = {e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7])};
    if (t >= hi) continue;
    if (!is_v) {
      *reinterpret_cast<u32x2*>(out + static_cast<size_t>(t) * D + d) = codes;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[(d + e) * (128 + 16) + t] = static_cast<uint8_t>(codes[e >> 2] >> (8 * (e & 3)));
    }
  }
  if (!is_v) return;
  __syncthreads();
  // 16 tokens of one dimension per store where all of them are new
  const int g0 = lo / 16, groups = (hi + 15) / 16 - g0;
  for (int i = threadIdx.x; i < groups * D; i += kThreads) {
    const int d = i / groups, g = g0 + i - d * groups;
    const uint8_t* const src = tile + d * (128 + 16) + 16 * g;
    uint8_t* const dst = out + static_cast<size_t>(d) * c.page + 16 * g;
    if (16 * g >= lo && 16 * g + 16 <= hi) {
      *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
    } else {
      const int from = max(lo - 16 * g, 0), to = min(hi - 16 * g, 16);
      for (int e = from; e < to; ++e) dst[e] = src[e];
    }
  }
}

// Pages that hold a sequence's new tokens, wherever the first one falls.
int page_span(const Kv8Cache& c) {
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  return (most + c.page - 2) / c.page + 1;
}

template <int D, bool kBf16>
hipError_t launch_dim(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                      hipStream_t stream) {
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int span = page_span(c);
  const int64_t blocks = kv8_append_blocks(c);
  if (blocks >= (int64_t{1} << 24)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(blocks)), block(kThreads);
  // a call of few tokens per sequence never fills a page: its rows need fewer registers
  const int rows = most < c.page ? most : c.page;
  const int chunks = rows * (D / 8);
#define MQ_APPEND(CPT)                                                                                            \
  return launch_kernel(kv8_append_kernel<D, CPT, kBf16>, grid, block, 0, stream, c, k, v, k_stride, v_stride, span)
  if (chunks <= kThreads) MQ_APPEND(1);
  if (chunks <= 2 * kThreads) MQ_APPEND(2);
  if (chunks <= 4 * kThreads) MQ_APPEND(4);
  MQ_APPEND(8);
#undef MQ_APPEND
}

}  // namespace

int64_t kv8_append_blocks(const Kv8Cache& c) { return static_cast<int64_t>(c.batch) * page_span(c) * c.kv_heads * 2; }

hipError_t launch_kv8_append(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                             int64_t v_stride, bool bf16, hipStream_t stream) {
  if (c.head_dim == 128)
    return bf16 ? launch_dim<128, true>(c, k, v, k_stride, v_stride, stream)
                : launch_dim<128, false>(c, k, v, k_stride, v_stride, stream);
  if (c.head_dim == 64)
    return bf16 ? launch_dim<64, true>(c, k, v, k_stride, v_stride, stream)
                : launch_dim<64, false>(c, k, v, k_stride, v_stride, stream);
  return hipErrorInvalidValue;
}

}  // namespace mq
