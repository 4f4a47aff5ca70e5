// What the attention kernels over the paged e4m3 KV cache share.
#pragma once

#include "block8_launch.h"
#include "device_common.h"

namespace mq {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_inff();
// Scales outside what the append writes would carry sums out of binary32.
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p120f;
// What the decode form's weights are raised by, as an exponent and as the
// factor that takes it back.
constexpr float kRaise = 15.f, kLower = 0x1p-15f;

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef float f32x8 __attribute__((ext_vector_type(8)));

// 8 e4m3 codes as 8 fp16 or bf16 values (exact).
template <bool kBf16>
__device__ __forceinline__ f16x8 widen(uint32_t lo, uint32_t hi) {
  if constexpr (kBf16) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    const u32x4 w = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                     __builtin_bit_cast(uint32_t, d)};
    return __builtin_bit_cast(f16x8, w);
  } else {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
}

__device__ __forceinline__ f16x8 to_f16(f32x8 v) { return __builtin_convertvector(v, f16x8); }

// 16 codes of which only the first n count: the others become 0.
__device__ __forceinline__ u32x4 first_bytes(u32x4 v, int n) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int k = n - 4 * w;
    v[w] = k >= 4 ? v[w] : k <= 0 ? 0u : v[w] & ((1u << (8 * k)) - 1u);
  }
  return v;
}

__device__ __forceinline__ float held_scale(float s) { return fminf(fmaxf(s, kMinScale), kMaxScale); }
// The logarithm of a held scale; a NaN, which held_scale hides, stays one here.
__device__ __forceinline__ float log_scale(float s) {
  const float l = __builtin_amdgcn_logf(held_scale(s));
  return s == s ? l : s;
}

// A sequence as the kernels see it.
struct Seq {
  int row0, n, len, seen;  // first row, new tokens, tokens, tokens that the table can hold
};

__device__ __forceinline__ Seq sequence(const Kv8Cache& c, int b) {
  Seq s;
  s.row0 = max(c.cu[b], 0);
  s.n = max(min(min(c.cu[b + 1], c.tokens) - s.row0, c.max_q_len), 0);
  s.len = c.lens[b];
  s.seen = static_cast<int>(min(static_cast<int64_t>(max(s.len, 0)), static_cast<int64_t>(c.table_width) * c.page));
  return s;
}

// Which of the 16 keys from new token `at` on (negative: before the new ones,
// where all are seen) a row's words name, the first in the lowest bit.
__device__ __forceinline__ uint32_t tree_bits(const int32_t* words, int count, int at) {
  if (at <= -16) return 0xffffu;
  const int k = at >> 5;
  const uint32_t lo = k < 0 ? 0xffffffffu : k < count ? static_cast<uint32_t>(words[k]) : 0u;
  const uint32_t hi = k + 1 < count ? static_cast<uint32_t>(words[k + 1]) : 0u;
  return static_cast<uint32_t>((static_cast<uint64_t>(hi) << 32 | lo) >> (at & 31)) & 0xffffu;
}
__device__ __forceinline__ uint32_t first_bits(int n) { return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Of 16 codes the NaN ones become 0 in v; returned are codes of 1 where they were.
__device__ __forceinline__ u32x4 take_nan(u32x4& v) {
  u32x4 ones;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t nan = (((v[w] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    v[w] &= ~(nan * 0xffu);
    ones[w] = nan * 0x38u;
  }
  return ones;
}
__device__ __forceinline__ bool has_any(u32x4 v) { return (v[0] | v[1] | v[2] | v[3]) != 0; }

// 8 fp16 values, 1 where the bit is set.
__device__ __forceinline__ f16x8 ones_of(uint32_t bits) {
  f16x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (bits >> e) & 1 ? static_cast<f16>(1.f) : static_cast<f16>(0.f);
  return v;
}

// The workspace of a split call: for every split and row (token, head) its
// maximum and sum, then its unnormalised output.
struct Parts {
  float* ml;  // [splits, rows, 2]
  float* o;   // [splits, rows, head_dim]
  // of shared-out trees [shares, kPromptRows] rows, the shares of a row tile kv_heads
  // apart, and for every row (token, head) the first one's and how many there are
  size_t rows;
  u32x2* where;
};

// The larger of x in lanes l and l ^ 32, in both: the swap leaves the lower
// half's values in one register and the upper half's in the other. (Written
// out: the compiler drops the second result of the builtin.)
__device__ __forceinline__ float halves_max(float x) {
  float lower = x, upper = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(lower), "+v"(upper));
  return fmaxf(lower, upper);
}

// The prompt and tree forms' reference of the exponentials follows the maximum
// lazily: it moves when a score passes it by more than 2^kLazy.
constexpr float kLazy = 4.f, kLazyRaise = kRaise - kLazy, kLazyLower = 0x1p-11f;

}  // namespace mq
