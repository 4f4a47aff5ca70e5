// Device helpers shared by the kernels that turn binary32 values into 8-bit
// codes under a scale: symmetric int8 and 8-bit floating point (OCP e4m3).
#pragma once

#include "device_common.h"

namespace mq {

// Distance from a half-integer below which an int8 code takes the IEEE
// division (see int8_codes).
constexpr float kTieMargin = 1.0f / 4096.0f;

// The reciprocal int8_codes multiplies by: rcp(s) for a normal s; infinity
// for a binary32-subnormal s (then every product is non-finite and each
// element takes the division).
__device__ __forceinline__ float code_rcp(float s) {
  return s < 1.17549435e-38f ? __builtin_inff() : __builtin_amdgcn_rcpf(s);
}

// Codes of 8 values as 8 bytes: rne(fl32(v / s)) for s > 0, clamped to
// [-127, 127]; 0 for s = 0. Each element forms
// u = rint(v * r + 128) with one fused multiply-add (r = rcp(s), within 1 ulp
// of 1/s). The product differs from the exact quotient v / s by at most 2^-22
// relative (< 3.1e-5 for quotients up to 127.5), the rounded sum adds at most
// 2^-17, and the correctly rounded quotient is within half an ulp (< 3.9e-6)
// of the exact one. So when v * r + 128 is more than kTieMargin away from
// every half-integer, the rounded quotient lies on the same side of the
// nearest half-integer and u - 128 is its code; the rest (about 1 element in
// 2000, and every non-finite product) take the IEEE division, whose correctly
// rounded result decides ties. Codes in [-127, 127] are u in [1, 255]; one
// unsigned 8-bit conversion per element packs u, and flipping bit 7 of each
// byte gives the two's-complement code u - 128.
__device__ __forceinline__ u32x2 int8_codes(const float (&f)[8], float s, float r) {
  if (!(s > 0.f)) return u32x2{0u, 0u};
  float u[8];
  bool slow = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = fmaf(f[e], r, 128.f);
    u[e] = rintf(p);
    slow |= !(fabsf(p - u[e]) <= 0.5f - kTieMargin);
  }
  if (slow) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = fmaf(f[e], r, 128.f);
      if (!(fabsf(p - u[e]) <= 0.5f - kTieMargin)) u[e] = rintf(f[e] / s) + 128.f;
    }
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e >> 2] = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_amdgcn_fmed3f(u[e], 1.f, 255.f), e & 3, w[e >> 2]);
  return u32x2{w[0] ^ 0x80808080u, w[1] ^ 0x80808080u};
}

constexpr float kE4m3Max = 448.f;

// Four binary32 values (each within +-448) rounded to nearest even as e4m3,
// element 0 in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

// e4m3 codes of 8 values as 8 bytes: rne(clamp(fl32(v / s), -448, 448)) for
// s > 0, 0 for s = 0. With r = rcp(s) the product p = v * r is within 2^-21
// relative of the correctly rounded quotient, and rounding to e4m3 is
// monotone: where p (1 - 2^-20) and p (1 + 2^-20) have the same code, that is
// the quotient's. Only where they differ (about 1 element in 60000 beside
// exact ties), or for a scale too small for a finite reciprocal product, the
// lane forms the IEEE quotients. s is at least max|v| / 448 up to rounding,
// so p stays within 448 (1 + 2^-20), which still rounds to 448.
__device__ __forceinline__ u32x2 e4m3_codes(const float (&f)[8], float s, float r) {
  if (!(s > 0.f)) return u32x2{0u, 0u};
  constexpr float kLo = 1.f - 0x1p-20f, kHi = 1.f + 0x1p-20f;
  u32x2 out;
  bool slow = s < 0x1p-100f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = f[4 * w + e] * r;
    const uint32_t lo = e4m3x4(p[0] * kLo, p[1] * kLo, p[2] * kLo, p[3] * kLo);
    const uint32_t hi = e4m3x4(p[0] * kHi, p[1] * kHi, p[2] * kHi, p[3] * kHi);
    out[w] = lo;
    slow |= lo != hi;
  }
  if (slow) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = __builtin_amdgcn_fmed3f(f[4 * w + e] / s, -kE4m3Max, kE4m3Max);
      out[w] = e4m3x4(q[0], q[1], q[2], q[3]);
    }
  }
  return out;
}

// Maximum over each row of 16 lanes, the same value in every lane of the row.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));   // quad_perm [1, 0, 3, 2]
  v = fmaxf(v, dpp_f32<0x4E>(v));   // quad_perm [2, 3, 0, 1]
  v = fmaxf(v, dpp_f32<0x141>(v));  // row_half_mirror
  return fmaxf(v, dpp_f32<0x140>(v));  // row_mirror
}

}  // namespace mq
