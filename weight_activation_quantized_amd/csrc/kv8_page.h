// Scales and codes of a page of the e4m3 KV cache, for the kernels that write one.
#pragma once

#include "device_common.h"
#include "quant_codes.h"

namespace mq {

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

constexpr uint32_t kNanCode = 0x7f;

// The four codes of a word times ratio, rounded to e4m3 again; NaN stays as it is.
__device__ __forceinline__ uint32_t moved(uint32_t w, float ratio) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  const uint32_t to = e4m3x4(clamp448(a[0] * ratio), clamp448(a[1] * ratio), clamp448(b[0] * ratio), clamp448(b[1] * ratio));
  // bytes of seven ones below the sign: adding 1 carries into the sign's place
  const uint32_t nan = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
  const uint32_t keep = nan * 0xffu;
  return (to & ~keep) | (w & keep);
}

}  // namespace mq
