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
// in place. A workgroup of q owns (sequence, as many tokens as a page has,
// query head). A thread reads the 8 values that its own 8 rotate with as well
// (half the head away; L1 has them), so no lane waits for another but for the
// norm's sum, which 16 or 8 lanes form by DPP in binary64. All in binary32,
// every product and sum rounded by itself, so that codes are defined bit for
// bit; q is rounded once.
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

// Sum over the D / 8 neighbouring lanes that hold a row, in each of them.
template <int D>
__device__ __forceinline__ double row_sum(double v) {
  v += dpp_f64<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp_f64<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp_f64<0x141>(v);  // row_half_mirror
  if constexpr (D == 128) v += dpp_f64<0x140>(v);  // row_mirror
  return v;
}

template <bool kBf16>
__device__ __forceinline__ void to_floats(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) word_to_floats<kBf16>(w[e], f[2 * e], f[2 * e + 1]);
}

// What a thread needs of the rotation for its 8 dimensions, whatever the token:
// where the values lie that rotate with its own, and the norm's weights of both.
template <bool kBf16>
struct Lane {
  int d, mate;  // its dimensions; those of the other half of its pairs (d itself where none are needed)
  float w[8], mate_w[8];
  __device__ __forceinline__ Lane(const Kv8Turn& t, const uint16_t* weight, int dim) : d(dim), mate(dim) {
    const int half = t.rot / 2;
    if (!t.next && d < t.rot) mate = d < half ? d + half : d - half;
    if (weight) {
      to_floats<kBf16>(*reinterpret_cast<const u32x4*>(weight + d), w);
      to_floats<kBf16>(*reinterpret_cast<const u32x4*>(weight + mate), mate_w);
    }
  }
};

// 8 values x of a token's head and their mates, normed and rotated. Every lane
// of a row takes part.
template <int D, bool kBf16>
__device__ __forceinline__ void turn(const Kv8Turn& t, const Lane<kBf16>& at, bool norm, u32x4 x, u32x4 mate, int pos,
                                     float (&f)[8]) {
#pragma clang fp contract(off)
  to_floats<kBf16>(x, f);
  float m[8];
  to_floats<kBf16>(mate, m);
  if (norm) {
    double sum = 0.;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += static_cast<double>(f[e]) * static_cast<double>(f[e]);
    const float r = static_cast<float>(1.0 / sqrt(row_sum<D>(sum) / D + t.eps));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = (f[e] * r) * at.w[e];
      m[e] = (m[e] * r) * at.mate_w[e];
    }
  }
  if (at.d >= t.rot) return;
  const int half = t.rot / 2;
  const bool known = static_cast<uint32_t>(pos) < static_cast<uint32_t>(t.max_pos);
  const float* const row = t.cos_sin + static_cast<int64_t>(known ? pos : 0) * t.rot;
  const float none = __builtin_nanf("");
  if (t.next) {
    const f32x4 c = *reinterpret_cast<const f32x4*>(row + at.d / 2), s = *reinterpret_cast<const f32x4*>(row + half + at.d / 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = f[2 * e], b = f[2 * e + 1], ce = known ? c[e] : none;
      f[2 * e] = a * ce - b * s[e];
      f[2 * e + 1] = b * ce + a * s[e];
    }
    return;
  }
  const bool upper = at.d >= half;
  const int i = upper ? at.mate : at.d;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const f32x4 c = *reinterpret_cast<const f32x4*>(row + i + 4 * q), s = *reinterpret_cast<const f32x4*>(row + half + i + 4 * q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // (x - y and x + -y are the same, bit for bit)
      const float ce = known ? c[e] : none, se = upper ? s[e] : -s[e];
      f[4 * q + e] = f[4 * q + e] * ce + m[4 * q + e] * se;
    }
  }
}

// The rows of one query head and as many tokens as a page has.
template <int D, int kThreads, int CPT, bool kBf16>
__device__ __forceinline__ void turn_queries(const Kv8Cache& c, const Kv8Turn& t, int b, int tile, int head) {
  constexpr int kDc = D / 8;
  const int first_row = max(c.cu[b], 0), n = min(min(c.cu[b + 1], c.tokens) - first_row, c.max_q_len);
  const int t0 = tile * c.page, count = min(n - t0, c.page);
  if (count <= 0) return;
  const int start = c.lens[b] - (c.cu[b + 1] - c.cu[b]);
  const Lane<kBf16> lane(t, t.q_weight, 8 * (static_cast<int>(threadIdx.x) % kDc));
  u32x4 x[CPT], mate[CPT];
  int pos[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int at = (static_cast<int>(threadIdx.x) + kThreads * i) / kDc;
    x[i] = mate[i] = u32x4{0u, 0u, 0u, 0u};
    pos[i] = 0;
    if (at < count) {
      const int64_t row = first_row + t0 + at;
      const uint16_t* const from = t.q + row * t.q_stride + head * D;
      x[i] = *reinterpret_cast<const u32x4*>(from + lane.d);
      mate[i] = *reinterpret_cast<const u32x4*>(from + lane.mate);
      pos[i] = t.positions ? t.positions[row] : start + t0 + at;
    }
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int at = (static_cast<int>(threadIdx.x) + kThreads * i) / kDc;
    float f[8];
    turn<D, kBf16>(t, lane, t.q_weight != nullptr, x[i], mate[i], pos[i], f);
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = half_bits<kBf16>(f[2 * e]) | (static_cast<uint32_t>(half_bits<kBf16>(f[2 * e + 1])) << 16);
    // (in place too: what this wavefront rotates was read above, and no other reads it)
    if (at < count)
      *reinterpret_cast<u32x4*>(t.q_out + (first_row + t0 + at) * t.q_out_stride + head * D + lane.d) = w;
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
  __shared__ __attribute__((aligned(16))) uint8_t tile[(kThreads == 64 ? kSmallPage : D * 128) + D / 8 * 16];

  // blockIdx.x = ((sequence * span + page) * kv_heads + head) * 2 + (0: K, 1: V),
  // with the rotation the query heads behind a page's kv heads
  unsigned at = blockIdx.x;
  unsigned unit_of_page = 0;
  if constexpr (kTurn) {
    const unsigned units = 2 * c.kv_heads + turning.q_heads;
    unit_of_page = at % units;
    at /= units;
    if (unit_of_page >= 2u * c.kv_heads) {
      turn_queries<D, kThreads, CPT, kBf16>(c, turning, static_cast<int>(at / span), static_cast<int>(at % span),
                                            static_cast<int>(unit_of_page) - 2 * c.kv_heads);
      return;
    }
  }
  const bool is_v = (kTurn ? unit_of_page : at) & 1;
  if constexpr (!kTurn) at >>= 1;
  const int head = static_cast<int>(kTurn ? unit_of_page >> 1 : at % c.kv_heads);
  if constexpr (!kTurn) at /= c.kv_heads;
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
  // The largest finite magnitude, and whether some value of this thread is not
  // finite. Rotated keys are binary32 values from here on.
  const bool turned_k = kTurn && !is_v;
  float f[kTurn ? CPT : 1][8];
  float amax;
  bool odd = false;
  if (turned_k) {
    if constexpr (kTurn) {
      const Lane<kBf16> lane(turning, turning.k_weight, d);
      u32x4 mate[CPT];
      int pos[CPT];
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int t = token(i);
        const int64_t row = row0 + t;
        mate[i] = u32x4{0u, 0u, 0u, 0u};
        pos[i] = 0;
        if (t >= lo && t < hi && row >= 0 && row < c.tokens) {
          mate[i] = *reinterpret_cast<const u32x4*>(x + row * stride + head * D + lane.mate);
          pos[i] = turning.positions ? turning.positions[row] : static_cast<int>(pos0) + t;
        }
      }
      if (!known) return;
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        turn<D, kBf16>(turning, lane, turning.k_weight != nullptr, w[i], mate[i], pos[i], f[i]);
        const bool mine = token(i) >= lo && token(i) < hi;  // (others' rotated zeros may be NaN)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t m = mine ? __builtin_bit_cast(uint32_t, f[i][e]) & 0x7fffffffu : 0u;
          odd |= m >= 0x7f800000u;
          most = m < 0x7f800000u ? max(most, m) : most;
        }
      }
      amax = __builtin_bit_cast(float, most);
    }
  } else {
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
  u32x2 codes[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float a[8];
    if constexpr (kTurn) {
      if (turned_k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = f[i][e];
      } else {
        to_floats<kBf16>(w[i], a);
      }
    } else {
      to_floats<kBf16>(w[i], a);
    }
    uint32_t bad = 0;
    if (odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        bad |= static_cast<uint32_t>((__builtin_bit_cast(uint32_t, a[e]) & 0x7fffffffu) >= 0x7f800000u) << e;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = quotient(a[e]);
    codes[i] = u32x2{e4m3x4(a[0], a[1], a[2], a[3]), e4m3x4(a[4], a[5], a[6], a[7])};
    if (odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t at = 8 * (e % 4);
        if ((bad >> e) & 1) codes[i][e / 4] = (codes[i][e / 4] & ~(0xffu << at)) | (kNanCode << at);
      }
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

template <int D, bool kBf16, bool kTurn>
hipError_t launch_dim(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                      const Kv8Turn& turning, hipStream_t stream) {
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int span = page_span(c);
  const int64_t blocks = kTurn ? kv8_rope_append_blocks(c, turning.q_heads) : kv8_append_blocks(c);
  if (blocks >= (int64_t{1} << 24)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(blocks));
  // A call of few tokens per sequence never fills a page: its rows need fewer
  // registers, and with little to move in a page one wavefront does (64
  // sequences of one token, pages of 16: 4.0 us, with four wavefronts 4.5).
  // Three more tokens where threads take four at a time.
  const int rows = most < c.page ? most : c.page;
  const int chunks = rows * (D / 8), padded = (rows + 3 < c.page ? rows + 3 : c.page) * (D / 8);
#define MQ_APPEND(TH, CPT)                                                                                          \
  return launch_kernel(kv8_append_kernel<D, TH, CPT, kBf16, kTurn>, grid, dim3(TH), 0, stream, c, k, v, k_stride, \
                       v_stride, span, turning)
  if (chunks <= 64 && c.page * D <= kSmallPage) MQ_APPEND(64, 1);
  if (chunks <= 256) MQ_APPEND(256, 1);
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
int64_t kv8_rope_append_blocks(const Kv8Cache& c, int q_heads) {
  return static_cast<int64_t>(c.batch) * page_span(c) * (c.kv_heads * 2 + q_heads);
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
