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
// With the rotation (kTurn) the same launch also norms q and k per head where
// weights are given, and rotates both by their positions' row of a table of
// cosines and sines: K on its way into the pages, q into a tensor of its own or
// in place. A lane has two pieces of 8 dimensions that rotate with each other, so
// nothing is exchanged but the norm's sum, which the 8 or 4 lanes of a row form by
// DPP in binary64. All in binary32, every product and sum rounded by itself, so
// that codes are defined bit for bit (the norm's factor but next to a rounding
// border: 127 additions and the root are off by 2^-46 at most); q is rounded once. 3 x 2048 tokens, 32 query
// heads on 8 of 128, with norms: 31.5 us, 4.0 TB/s (q alone 22, k and v alone 16);
// 64 sequences of one token 4.7, 3.5 of it the launch and q's loads.
//
// Bound by latency (lengths, page, rows, maximum, codes follow from each other)
// for few tokens, 4.0 us for 64 sequences of one; for prompts by that and HBM:
// 3 x 2048 tokens of 8 heads of 128 take 10.6 us, 3.2 TB/s (single codes into
// unpadded LDS, 16 lanes on one bank, and IEEE divisions took 1.55 times as
// long). Times in this file: captured calls one after the other, over three
// sets of inputs in turn.
#include "block8_launch.h"
#include "device_common.h"
#include "kv8_page.h"
#include "quant_codes.h"

namespace mq {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// The bytes of four words as columns: byte e of word t becomes byte t of out[e].
__device__ __forceinline__ void turned(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400);
  const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
  out[0] = __builtin_amdgcn_perm(b, a, 0x05040100);
  out[1] = __builtin_amdgcn_perm(b, a, 0x07060302);
  out[2] = __builtin_amdgcn_perm(d, c, 0x05040100);
  out[3] = __builtin_amdgcn_perm(d, c, 0x07060302);
}

// A double from another lane of the same 16, by DPP control kCtrl.
template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double x) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  const u32x2 r = {static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b[0]), kCtrl, 0xF, 0xF, false)),
                   static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b[1]), kCtrl, 0xF, 0xF, false))};
  return __builtin_bit_cast(double, r);
}

// Sum over the D / 16 neighbouring lanes that hold a row, in each of them.
template <int D>
__device__ __forceinline__ double row_sum(double v) {
  v += dpp_f64<0xB1>(v);  // quad_perm [1, 0, 3, 2]
  v += dpp_f64<0x4E>(v);  // quad_perm [2, 3, 0, 1]
  if constexpr (D == 128) v += dpp_f64<0x141>(v);  // row_half_mirror
  return v;
}

// Two binary32 values rounded to 16 bits, the first in the lower half.
template <bool kBf16>
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  if constexpr (kBf16) return bf16x2_bits(lo, hi);
  return as_u32(__builtin_convertvector(f32x2{lo, hi}, f16x2));
}

template <bool kBf16>
__device__ __forceinline__ void to_floats(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) word_to_floats<kBf16>(w[e], f[2 * e], f[2 * e + 1]);
}

// The two pieces of 8 dimensions of a head that lane k of its D / 16 has: such that
// rotate with each other, or where nothing rotates or neighbours do any two.
struct Pieces {
  int d[2];
  __device__ __forceinline__ Pieces(const Kv8Turn& t, int k) {
    const int half = t.rot / 2;
    if (!t.next && 8 * k < half) {
      d[0] = 8 * k;
      d[1] = 8 * k + half;
    } else {
      d[0] = 16 * k;
      d[1] = 16 * k + 8;
    }
  }
};

// Cosines and sines of a token's position for those pieces (NaN: no such position).
struct Angles {
  f32x4 c[2], s[2];  // pairs half a head apart: 8 of each; neighbours: 4 for each piece
  __device__ __forceinline__ void load(const Kv8Turn& t, const Pieces& at, int pos) {
    const int half = t.rot / 2;
    if (at.d[0] >= t.rot) return;
    const bool known = static_cast<uint32_t>(pos) < static_cast<uint32_t>(t.max_pos);
    const float* const row = t.cos_sin + static_cast<int64_t>(known ? pos : 0) * t.rot + (t.next ? at.d[0] / 2 : at.d[0]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      c[q] = *reinterpret_cast<const f32x4*>(row + 4 * q);
      s[q] = *reinterpret_cast<const f32x4*>(row + half + 4 * q);
    }
    if (!known) {
      const float none = __builtin_nanf("");
      c[0] = c[1] = f32x4{none, none, none, none};
    }
  }
};

// 1 / sqrt(m) within 2^-50 of itself: the instruction's estimate and two steps of
// Newton's iteration (a square root and a division take four times as long).
__device__ __forceinline__ double inverse_root(double m) {
#pragma clang fp contract(fast)
  const double y0 = __builtin_amdgcn_rsq(m);
  double y = y0;
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(y * 0.5, fma(-(m * y), y, 1.0), y);
  return m > 0.0 && m < __builtin_inf() ? y : y0;  // (0 for infinity, infinity for 0, NaN)
}

// Two pieces x of a token's head, normed (w: the weights of both) and rotated.
// Every lane of a row takes part.
template <int D, bool kBf16>
__device__ __forceinline__ void turn(const Kv8Turn& t, const Pieces& at, const u32x4 (&w)[2], bool norm,
                                     const u32x4 (&x)[2], const Angles& angle, float (&f)[2][8]) {
#pragma clang fp contract(off)
  to_floats<kBf16>(x[0], f[0]);
  to_floats<kBf16>(x[1], f[1]);
  if (norm) {
    double sum = 0.;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += static_cast<double>(f[q][e]) * static_cast<double>(f[q][e]);
    const float r = static_cast<float>(inverse_root(row_sum<D>(sum) / D + t.eps));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float g[8];
      to_floats<kBf16>(w[q], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[q][e] = (f[q][e] * r) * g[e];
    }
  }
  if (at.d[0] >= t.rot) return;
  if (t.next) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = f[q][2 * e], b = f[q][2 * e + 1];
        f[q][2 * e] = a * angle.c[q][e] - b * angle.s[q][e];
        f[q][2 * e + 1] = b * angle.c[q][e] + a * angle.s[q][e];
      }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = f[0][e], b = f[1][e], c = angle.c[e / 4][e % 4], s = angle.s[e / 4][e % 4];
      f[0][e] = a * c - b * s;
      f[1][e] = b * c + a * s;
    }
  }
}

// Queries: a workgroup takes `tile` tokens of a sequence (a power of two) and
// `heads_of` query heads, D / 16 lanes a row; lanes beyond the tokens take other
// heads. A token's angles are read once for all heads of its lanes, four heads'
// values are on their way at a time.
template <int D, int kThreads, bool kBf16>
__device__ __forceinline__ void turn_queries(const Kv8Cache& c, const Kv8Turn& t, int b, int tile, int part) {
  constexpr int kL = D / 16, kAtOnce = kThreads == 64 ? 2 : 4;
  const int first_row = max(c.cu[b], 0), n = min(min(c.cu[b + 1], c.tokens) - first_row, c.max_q_len);
  if (tile * t.tile >= n) return;
  const int start = c.lens[b] - (c.cu[b + 1] - c.cu[b]);
  const int slot = static_cast<int>(threadIdx.x) / kL, token = tile * t.tile + slot % t.tile;
  const int step = kThreads / kL / t.tile, end = min((part + 1) * t.heads_of, t.q_heads);
  const bool live = token < n;
  const int64_t row = first_row + (live ? token : 0);
  const Pieces at(t, static_cast<int>(threadIdx.x) % kL);
  const bool norm = t.q_weight != nullptr;
  u32x4 w[2];
  if (norm) {
    w[0] = *reinterpret_cast<const u32x4*>(t.q_weight + at.d[0]);
    w[1] = *reinterpret_cast<const u32x4*>(t.q_weight + at.d[1]);
  }
  Angles angle;
  angle.load(t, at, t.positions ? t.positions[row] : start + token);
  const uint16_t* const from = t.q + row * t.q_stride;
  uint16_t* const to = t.q_out + row * t.q_out_stride;
  for (int h0 = part * t.heads_of + slot / t.tile; h0 < end; h0 += kAtOnce * step) {
    u32x4 x[kAtOnce][2];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        x[i][q] = *reinterpret_cast<const u32x4*>(from + min(h0 + i * step, end - 1) * D + at.d[q]);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      float f[2][8];
      turn<D, kBf16>(t, at, w, norm, x[i], angle, f);
      // (in place too: a row's lanes are of one wavefront, which has read it)
      if (live && h0 + i * step < end)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          u32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = half_pair<kBf16>(f[q][2 * e], f[q][2 * e + 1]);
          *reinterpret_cast<u32x4*>(to + (h0 + i * step) * D + at.d[q]) = v;
        }
    }
  }
}

constexpr int kSmallPage = 4096;  // bytes of a page's head that one wavefront takes at most

// CPT: 16-byte chunks (8 values) of a page's rows per thread. With four or more
// a thread of V takes them from four consecutive tokens (of the page: from a
// multiple of four), turns the 4 x 8 codes in registers and writes words to
// LDS; with fewer it writes single codes.
template <int D, int kThreads, int CPT, bool kBf16, bool kTurn>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Cache c, const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, int64_t k_stride,
                                                              int64_t v_stride, int span, Kv8Turn turning) {
  constexpr int kDc = D / 8;  // chunks per row
  __shared__ float wmax[kThreads / 64];
  constexpr bool kQuads = CPT % 4 == 0;
  // V of the page as [D, page], 16 bytes of padding after every 8 rows: lanes
  // that write the same token of rows 8 apart meet no bank twice
  // (not where few tokens are rotated: their V codes go out one by one)
  constexpr bool kDirect = kTurn && kThreads == 64;
  __shared__ __attribute__((aligned(16))) uint8_t tile[kDirect ? 16 : (kThreads == 64 ? kSmallPage : D * 128) + D / 8 * 16];

  // blockIdx.x = ((sequence * span + page) * kv_heads + head) * 2 + (0: K, 1: V),
  // with the rotation without the workgroups of the queries
  unsigned at = blockIdx.x;
  if constexpr (kTurn) {
    // Evenly among each other: those of the queries stream, those of the keys and
    // values wait for one load after the other (3 x 2048 tokens: 32.9 us, one kind
    // behind the other 36.5). Of few tokens the queries first (256 x 1: 8.7, else 10.7).
    const unsigned queries = static_cast<unsigned>(c.batch) * turning.tiles * turning.parts;
    const unsigned before = kThreads == 64 ? min(at, queries) : __umulhi(at, turning.share);
    const unsigned behind = kThreads == 64 ? min(at + 1, queries) : __umulhi(at + 1, turning.share);
    if (behind != before) {
      const unsigned tile = before / turning.parts;
      turn_queries<D, kThreads, kBf16>(c, turning, static_cast<int>(tile / turning.tiles),
                                       static_cast<int>(tile % turning.tiles), static_cast<int>(before % turning.parts));
      return;
    }
    at -= before;
  }
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
  // The largest finite magnitude, and whether some value of this thread is not
  // finite. Rotated keys are binary32 values from here on, two pieces of 8 that a
  // lane of the row has.
  const bool turned_k = kTurn && !is_v;
  constexpr int kL = D / 16, kPairs = kTurn ? (CPT + 1) / 2 : 1;
  float f[kPairs][2][8];
  u32x4 w[CPT];
  const Pieces pieces(turning, static_cast<int>(threadIdx.x) % kL);
  auto pair_token = [&](int i) { return lo + (static_cast<int>(threadIdx.x) + kThreads * i) / kL; };
  float amax;
  bool odd = false;
  if (turned_k) {
    if constexpr (kTurn) {
      const bool norm = turning.k_weight != nullptr;
      u32x4 weight[2], raw[kPairs][2];
      Angles angle[kPairs];
      if (norm) {
        weight[0] = *reinterpret_cast<const u32x4*>(turning.k_weight + pieces.d[0]);
        weight[1] = *reinterpret_cast<const u32x4*>(turning.k_weight + pieces.d[1]);
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int t = pair_token(i);
        const int64_t row = row0 + t;
        raw[i][0] = raw[i][1] = u32x4{0u, 0u, 0u, 0u};
        int pos = static_cast<int>(pos0) + t;
        if (t < hi && row >= 0 && row < c.tokens) {
          if (turning.positions) pos = turning.positions[row];
          raw[i][0] = *reinterpret_cast<const u32x4*>(x + row * stride + head * D + pieces.d[0]);
          raw[i][1] = *reinterpret_cast<const u32x4*>(x + row * stride + head * D + pieces.d[1]);
        }
        angle[i].load(turning, pieces, pos);
      }
      if (!known) return;
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        turn<D, kBf16>(turning, pieces, weight, norm, raw[i], angle[i], f[i]);
        const bool mine = pair_token(i) < hi;  // (zeros of the others may have become NaN)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t m = mine ? __builtin_bit_cast(uint32_t, f[i][e / 8][e % 8]) & 0x7fffffffu : 0u;
          odd |= m >= 0x7f800000u;
          most = m < 0x7f800000u ? max(most, m) : most;
        }
      }
      amax = __builtin_bit_cast(float, most);
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int t = token(i);
      const int64_t row = row0 + t;
      w[i] = u32x4{0u, 0u, 0u, 0u};
      if (t >= lo && t < hi && row >= 0 && row < c.tokens)
        w[i] = *reinterpret_cast<const u32x4*>(x + row * stride + head * D + d);
    }
    if (!known) return;  // (the page's number was on its way with the rows)
    // as 16-bit patterns, whose order is the values' (with infinity and NaN
    // above all others)
    constexpr uint32_t kInfinite = kBf16 ? 0x7f80 : 0x7c00;
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i][e] & 0x7fff7fffu));
    uint32_t most = max(static_cast<uint32_t>(top[0]), static_cast<uint32_t>(top[1]));
    odd = most >= kInfinite;
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
    float unused;
    word_to_floats<kBf16>(most, amax, unused);
  }
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
  // 8 codes; of values that are not finite (where some are) that of NaN.
  auto codes_of = [&](const float (&a)[8]) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = quotient(a[e]);
    u32x2 code = {e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7])};
    if (odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t at = 8 * (e % 4);
        if ((__builtin_bit_cast(uint32_t, a[e]) & 0x7fffffffu) >= 0x7f800000u)
          code[e / 4] = (code[e / 4] & ~(0xffu << at)) | (kNanCode << at);
      }
    }
    return code;
  };
  if (turned_k) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if (pair_token(i) >= hi) continue;
      uint8_t* const to = out + static_cast<size_t>(pair_token(i)) * D;
      *reinterpret_cast<u32x2*>(to + pieces.d[0]) = codes_of(f[i][0]);
      *reinterpret_cast<u32x2*>(to + pieces.d[1]) = codes_of(f[i][1]);
    }
    return;
  }
  u32x2 codes[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float a[8];
    to_floats<kBf16>(w[i], a);
    codes[i] = codes_of(a);
  }
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (token(i) < hi) *reinterpret_cast<u32x2*>(out + static_cast<size_t>(token(i)) * D + d) = codes[i];
    return;
  }
  if constexpr (kDirect) {
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (token(i) < hi)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          out[static_cast<size_t>(d + e) * c.page + token(i)] = static_cast<uint8_t>(codes[i][e >> 2] >> (8 * (e & 3)));
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

// With little to move in a page one wavefront does (64 sequences of one token,
// pages of 16: 4.0 us, with four wavefronts 4.5). With the rotation, whose rows
// take half as many lanes: up to 8 tokens of 128 dimensions (256 sequences of one
// token, pages of 64: 8.7 us, with four wavefronts 19.3), two for up to 16 (8 x 750
// tokens in pages of 16: 38 us, with four 48).
int append_threads(const Kv8Cache& c, bool turned) {
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int chunks = (most < c.page ? most : c.page) * (c.head_dim / 8);
  if (turned) return chunks <= 128 ? 64 : chunks <= 256 ? 128 : 256;
  return chunks <= 64 && c.page * c.head_dim <= kSmallPage ? 64 : 256;
}

template <int D, bool kBf16, bool kTurn>
hipError_t launch_dim(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                      const Kv8Turn& turning, hipStream_t stream) {
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int span = page_span(c);
  int64_t blocks = kv8_append_blocks(c);
  // A call of few tokens per sequence never fills a page: its rows need fewer
  // registers. Three more tokens where threads take four at a time.
  const int rows = most < c.page ? most : c.page;
  const int chunks = rows * (D / 8), padded = (rows + 3 < c.page ? rows + 3 : c.page) * (D / 8);
  const int threads = append_threads(c, kTurn);
  Kv8Turn t = turning;
  if constexpr (kTurn) {
    // in 1 / 2^32, up: floor(n share / 2^32) counts from 0 to the queries' workgroups
    // as n does to all (under 2^24 of them)
    const uint64_t queries = static_cast<uint64_t>(c.batch) * t.tiles * t.parts;
    blocks += static_cast<int64_t>(queries);
    t.share = static_cast<uint32_t>(((queries << 32) + blocks - 1) / blocks);
  }
  if (blocks >= (int64_t{1} << 24)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(blocks));
#define MQ_APPEND(TH, CPT)                                                                                          \
  return launch_kernel(kv8_append_kernel<D, TH, CPT, kBf16, kTurn>, grid, dim3(TH), 0, stream, c, k, v, k_stride, \
                       v_stride, span, t)
  if (threads == 64) {
    if constexpr (kTurn) {
      if (chunks > 64) MQ_APPEND(64, 2);
    }
    MQ_APPEND(64, 1);
  }
  if constexpr (kTurn) {
    if (threads == 128) MQ_APPEND(128, 2);
  } else {
    if (chunks <= 256) MQ_APPEND(256, 1);
  }
  if (chunks <= 512) MQ_APPEND(256, 2);
  if (padded <= 1024) MQ_APPEND(256, 4);
  MQ_APPEND(256, 8);
#undef MQ_APPEND
}

template <bool kTurn>
hipError_t launch(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                  const Kv8Turn& turning, bool bf16, hipStream_t stream) {
  if (c.head_dim == 128)
    return bf16 ? launch_dim<128, true, kTurn>(c, k, v, k_stride, v_stride, turning, stream)
                : launch_dim<128, false, kTurn>(c, k, v, k_stride, v_stride, turning, stream);
  if (c.head_dim == 64)
    return bf16 ? launch_dim<64, true, kTurn>(c, k, v, k_stride, v_stride, turning, stream)
                : launch_dim<64, false, kTurn>(c, k, v, k_stride, v_stride, turning, stream);
  return hipErrorInvalidValue;
}

}  // namespace

int64_t kv8_append_blocks(const Kv8Cache& c) { return static_cast<int64_t>(c.batch) * page_span(c) * c.kv_heads * 2; }

// Workgroups of the queries: as many tokens side by side as there are, the other
// lanes other heads; a multiple of four heads a lane, and workgroups enough for all
// compute units where heads allow it (3 x 2048 tokens, 32 heads: 31.5 us with about
// 2048 workgroups, 32.9 with 1024, 36.2 with 512; 512 tokens of one sequence 7.4,
// with lanes of any number of heads 8.9).
Kv8Turn plan_kv8_turn(const Kv8Cache& c, Kv8Turn t) {
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int slots = append_threads(c, true) / (c.head_dim / 16);
  for (t.tile = 1; t.tile < slots && t.tile < most;) t.tile *= 2;
  t.tiles = (most + t.tile - 1) / t.tile;
  const int side = slots / t.tile;  // heads side by side
  const int64_t rows = static_cast<int64_t>(c.batch) * t.tiles;
  const int64_t want = (2048 + rows - 1) / rows;  // parts of the heads
  int64_t each = (t.q_heads + want - 1) / want;
  each = (each + 4 * side - 1) / (4 * side) * (4 * side);
  t.heads_of = static_cast<int>(each);
  t.parts = (t.q_heads + t.heads_of - 1) / t.heads_of;
  return t;
}
int64_t kv8_rope_append_blocks(const Kv8Cache& c, const Kv8Turn& t) {
  return kv8_append_blocks(c) + static_cast<int64_t>(c.batch) * t.tiles * t.parts;
}

hipError_t launch_kv8_append(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                             int64_t v_stride, bool bf16, hipStream_t stream) {
  return launch<false>(c, k, v, k_stride, v_stride, Kv8Turn{}, bf16, stream);
}

hipError_t launch_kv8_rope_append(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                  int64_t v_stride, const Kv8Turn& turning, bool bf16, hipStream_t stream) {
  return launch<true>(c, k, v, k_stride, v_stride, turning, bf16, stream);
}

}  // namespace mq
