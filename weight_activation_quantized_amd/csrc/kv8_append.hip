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
// A NaN or infinity takes no part in a and becomes the code of NaN, which no
// change of scale touches: it spoils its own token and no other of the page.
//
// A workgroup owns one (sequence, page, head, K or V): the new rows of the
// page stay in registers between the maximum and the codes, so they are read
// once, and nothing is shared between workgroups (no atomics, the same bits
// every time). K rows go out as they come. V pages are stored transposed,
// [head_dim, page]: the attention's second product then reads 16 tokens of one
// dimension with one load; the transposition happens here, once per token, in
// registers and LDS.
//
// Bound by latency (lengths, page, rows, maximum, codes follow from each other)
// for few tokens, 4.0 us for 64 sequences of one; for prompts by that and HBM:
// 3 x 2048 tokens of 8 heads of 128 take 10.6 us, 3.2 TB/s (single codes into
// unpadded LDS, 16 lanes on one bank, and IEEE divisions took 1.55 times as
// long). Times in this file: captured calls one after the other, over three
// sets of inputs in turn.
#include "block8_launch.h"
#include "device_common.h"
#include "quant_codes.h"

namespace mq {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

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

// The bytes of four words as columns: byte e of word t becomes byte t of out[e].
__device__ __forceinline__ void turned(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400);
  const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
  out[0] = __builtin_amdgcn_perm(b, a, 0x05040100);
  out[1] = __builtin_amdgcn_perm(b, a, 0x07060302);
  out[2] = __builtin_amdgcn_perm(d, c, 0x05040100);
  out[3] = __builtin_amdgcn_perm(d, c, 0x07060302);
}

constexpr int kSmallPage = 4096;  // bytes of a page's head that one wavefront takes at most

// CPT: 16-byte chunks (8 values) of a page's rows per thread. With four or more
// a thread of V takes them from four consecutive tokens (of the page: from a
// multiple of four), turns the 4 x 8 codes in registers and writes words to
// LDS; with fewer it writes single codes.
template <int D, int kThreads, int CPT, bool kBf16>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Cache c, const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, int64_t k_stride,
                                                              int64_t v_stride, int span) {
  constexpr int kDc = D / 8;  // chunks per row
  __shared__ float wmax[kThreads / 64];
  constexpr bool kQuads = CPT % 4 == 0;
  // V of the page as [D, page], 16 bytes of padding after every 8 rows: lanes
  // that write the same token of rows 8 apart meet no bank twice
  __shared__ __attribute__((aligned(16))) uint8_t tile[(kThreads == 64 ? kSmallPage : D * 128) + D / 8 * 16];

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
  const bool known = id >= 0 && id < c.num_pages;
  const int lo = max(start - static_cast<int>(pos0), 0);                    // first new token of the page
  // behind the last (a sequence longer than max_q_len is cut to what the
  // registers hold, never read or written past them)
  const int hi = min(min(len - static_cast<int>(pos0), c.page), (kQuads ? lo & ~3 : lo) + CPT * kThreads / kDc);
  const int64_t row0 = first_row + pos0 - start;  // row of the page's token 0
  const size_t unit = static_cast<size_t>(known ? id : 0) * c.kv_heads + head;
  float* const scale_at = (is_v ? c.v_scales : c.k_scales) + unit;
  uint8_t* const out = (is_v ? c.v : c.k) + unit * c.page * D;
  const float old = lo > 0 ? *scale_at : 0.f;

  // Token and first dimension of this thread's chunk i.
  const bool quads = kQuads && is_v;
  auto token = [&](int i) {
    return quads ? (lo & ~3) + 4 * ((static_cast<int>(threadIdx.x) + kThreads * (i / 4)) / kDc) + i % 4
                 : lo + (static_cast<int>(threadIdx.x) + kThreads * i) / kDc;
  };
  const int d = 8 * (static_cast<int>(threadIdx.x) % kDc);  // (kDc divides kThreads)
  const uint16_t* const x = is_v ? v : k;
  const int64_t stride = is_v ? v_stride : k_stride;
  u32x4 w[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int t = token(i);
    const int64_t row = row0 + t;
    w[i] = u32x4{0u, 0u, 0u, 0u};
    if (t >= lo && t < hi && row >= 0 && row < c.tokens)
      w[i] = *reinterpret_cast<const u32x4*>(x + row * stride + head * D + d);
  }
  if (!known) return;  // (the page's number was on its way with the rows)
  // The largest magnitude, as 16-bit patterns, whose order is the values' (with
  // infinity and NaN above all others).
  constexpr uint32_t kInfinite = kBf16 ? 0x7f80 : 0x7c00;
  u16x2 top = {0, 0};
#pragma unroll
  for (int i = 0; i < CPT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i][e] & 0x7fff7fffu));
  uint32_t most = max(static_cast<uint32_t>(top[0]), static_cast<uint32_t>(top[1]));
  const bool odd = most >= kInfinite;  // some value of this thread is not finite
  if (odd) {
    most = 0;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = (w[i][e / 2] >> (16 * (e % 2))) & 0x7fffu;
        most = m < kInfinite ? max(most, m) : most;
      }
  }
  float amax, unused;
  word_to_floats<kBf16>(most, amax, unused);
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) amax = fmaxf(amax, wmax[i]);

  float s = page_scale(amax);
  if (lo > 0) {  // the page holds older tokens
    if (s > old) {
      const float ratio = old / s;
      // 16 bytes at a time, a thread's loads together: of K rows all bytes, of
      // V rows (one dimension, `page` tokens) those of tokens before lo; the
      // others keep theirs (new codes are written after the barrier)
      const int per = is_v ? (lo + 15) / 16 : D / 16, all = (is_v ? D : lo) * per, pitch = is_v ? c.page : D;
      constexpr int kAtOnce = CPT >= 4 ? 2 : 4;
      for (int i0 = threadIdx.x; i0 < all; i0 += kAtOnce * kThreads) {
        int at[kAtOnce], keep[kAtOnce];
        u32x4 v[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          const int i = min(i0 + e * kThreads, all - 1), row = i / per, col = i - row * per;
          at[e] = row * pitch + 16 * col;
          keep[e] = i0 + e * kThreads < all ? (is_v ? min(lo - 16 * col, 16) : 16) : 0;
          v[e] = *reinterpret_cast<const u32x4*>(out + at[e]);
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          if (keep[e] == 0) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = min(max(keep[e] - 4 * q, 0), 4);
            const uint32_t mask = k == 4 ? 0xffffffffu : (1u << (8 * k)) - 1u;
            v[e][q] = (moved(v[e][q], ratio) & mask) | (v[e][q] & ~mask);
          }
          *reinterpret_cast<u32x4*>(out + at[e]) = v[e];
        }
      }
    } else {
      s = old;
    }
  }
  __syncthreads();  // every lane has read the old scale, and older codes are in place
  if (threadIdx.x == 0) *scale_at = s;

  // x / s. The scales that this kernel makes are powers of two of normal
  // reciprocal: their product is the quotient, bit for bit (one exact scaling
  // and at most one rounding in both). Others may stand in a cache that was
  // filled otherwise.
  const uint32_t sb = __builtin_bit_cast(uint32_t, s);
  const bool simple = (sb & 0x7fffffu) == 0 && sb >= 0x01000000u && sb <= 0x7e000000u;
  const float r = 1.f / s;
  auto quotient = [&](float a) { return clamp448(simple ? a * r : a / s); };
  u32x2 codes[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, z;
      word_to_floats<kBf16>(w[i][e], a, z);
      f[2 * e] = quotient(a);
      f[2 * e + 1] = quotient(z);
    }
    codes[i] = u32x2{e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7])};
  }
  if (odd) {
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = (w[i][e / 2] >> (16 * (e % 2))) & 0x7fffu, at = 8 * (e % 4);
        if (m >= kInfinite) codes[i][e / 4] = (codes[i][e / 4] & ~(0xffu << at)) | (kNanCode << at);
      }
  }
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (token(i) < hi) *reinterpret_cast<u32x2*>(out + static_cast<size_t>(token(i)) * D + d) = codes[i];
    return;
  }
  uint8_t* const rows = tile + d * c.page + 2 * d;  // (16 bytes for every 8 rows)
  if constexpr (kQuads) {
#pragma unroll
    for (int i = 0; i < CPT; i += 4) {
      const int t = token(i);
      if (t >= hi) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t in[4] = {codes[i][p], codes[i + 1][p], codes[i + 2][p], codes[i + 3][p]};
        uint32_t turn[4];
        turned(in, turn);
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(rows + (4 * p + e) * c.page + t) = turn[e];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int t = token(i);
      if (t >= hi) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) rows[e * c.page + t] = static_cast<uint8_t>(codes[i][e >> 2] >> (8 * (e & 3)));
    }
  }
  __syncthreads();
  // 16 tokens of one dimension per store where all of them are new
  const int g0 = lo / 16, groups = (hi + 15) / 16 - g0;
  for (int i = threadIdx.x; i < groups * D; i += kThreads) {
    const int row = i / groups, g = g0 + i - row * groups;
    const uint8_t* const src = tile + row * c.page + 16 * (row / 8) + 16 * g;
    uint8_t* const dst = out + static_cast<size_t>(row) * c.page + 16 * g;
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
  const dim3 grid(static_cast<uint32_t>(blocks));
  // A call of few tokens per sequence never fills a page: its rows need fewer
  // registers, and with little to move in a page one wavefront does (64
  // sequences of one token, pages of 16: 4.0 us, with four wavefronts 4.5).
  // Three more tokens where threads take four at a time.
  const int rows = most < c.page ? most : c.page;
  const int chunks = rows * (D / 8), padded = (rows + 3 < c.page ? rows + 3 : c.page) * (D / 8);
#define MQ_APPEND(TH, CPT)                                                                                         \
  return launch_kernel(kv8_append_kernel<D, TH, CPT, kBf16>, grid, dim3(TH), 0, stream, c, k, v, k_stride, v_stride, \
                       span)
  if (chunks <= 64 && c.page * D <= kSmallPage) MQ_APPEND(64, 1);
  if (chunks <= 256) MQ_APPEND(256, 1);
  if (chunks <= 512) MQ_APPEND(256, 2);
  if (padded <= 1024) MQ_APPEND(256, 4);
  MQ_APPEND(256, 8);
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
