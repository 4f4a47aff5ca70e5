// Causal attention over the paged e4m3 KV cache, for gfx950: single new tokens
// (decode) and prompts.
//
//   o[row] = sum_t p_t v_t,  p = softmax over the keys t <= position of the row
//   of softmax_scale * (q . k_t),  k_t = code * k_scale(page, head), v_t likewise
//
// Both forms compute S^T = K Q^T and O^T = V^T P^T: a lane of the result then
// holds one query row (its maximum and sum are lane values), and S^T's
// registers are, as they stand, the B operand of the second product. That
// needs two free choices. Which token a row of the K tile is can be chosen
// (each lane just reads another row of the page), and it is chosen so that a
// lane's scores belong to consecutive tokens. And V pages are stored
// transposed, so that the 8 or 16 consecutive tokens of one dimension that a
// lane needs are one load.
//
// Codes are widened exactly: K to the type of q, V to fp16. Scores and their
// statistics are binary32. The page's V scale joins the exponent: with
//   x_t = score_t log2(e) + log2(v_scale_t),   m = max x_t,   w_t = 2^(x_t - m + 15)
// the second product is sum w_t code_t in units of 2^(m - 15) whatever the
// scales of the pages are, and the sum of the weights is 2^-15 sum w_t / v_scale_t.
// w is rounded once, to fp16 (11 bits; bf16 would lose three more). The 2^15
// puts the largest weight at the top of fp16's range: with weights of at most 1
// those 2^-25 below the largest were lost to the output, though the sum counted
// them (one key of weight 0.999 and value 0 before 32767 others, which then are
// the whole output: nothing of it was left). Now that is 2^-40, in prompts (whose
// reference follows the maximum lazily) 2^-36.
//
// Keys that a row does not see get the weight 0 by a select, and V codes
// behind the last token are cleared, so whatever a page holds there (NaN codes
// too) counts for nothing; so do pages whose number is not one of the pool's.
// A row that sees no key is 0.
#include <type_traits>

#include "block8_launch.h"
#include "device_common.h"

namespace mq {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_inff();
// Scales outside what the append writes would carry sums out of binary32.
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p120f;
// What the decode form's weights are raised by, as an exponent and as the
// factor that takes it back.
constexpr float kRaise = 15.f, kLower = 0x1p-15f;

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

// Tiles of 64 keys that split `z` of `splits` takes of a sequence: [first,
// first + count). Every split gets the same number, at least `least`.
struct Span {
  int first, end;
};
__device__ __forceinline__ Span tiles_of(int tiles, int splits, int z, int least) {
  const int per = max((tiles + splits - 1) / splits, least);
  Span s;
  s.first = min(static_cast<int>(min(static_cast<int64_t>(z) * per, static_cast<int64_t>(tiles))), tiles);
  s.end = min(s.first + per, tiles);
  return s;
}

// The workspace of a split call: for every split and row (token, head) its
// maximum and sum, then its unnormalised output.
struct Parts {
  float* ml;  // [splits, rows, 2]
  float* o;   // [splits, rows, head_dim]
};

// ---------------------------------------------------------------------------
// Decode: the rows of one kv head (its query heads times the new tokens) stand
// in tiles of 16. A workgroup of four or eight wavefronts takes one such tile
// and a range of keys, a wavefront every fourth or eighth tile of 64 keys. Bound by the cache
// read: K and V go from memory straight into registers (16-byte loads, whole
// 64-byte pieces of a page row), K of the next tile is requested as soon as
// this tile's scores are formed, V as soon as its product is, and several
// wavefronts per SIMD keep the loads of a compute unit outstanding.
// v_mfma_16x16x32: lane (i = lane % 16, h = lane / 16). Row i of K tile j is
// token 16 (i / 4) + 4 j + i % 4, so lane (i, h) ends up with the scores of
// row i of Q for tokens 16 h .. 16 h + 15, in order.
//
// 64 sequences of up to 8193 keys, 32 query heads on 8 of 128: 135 us with the
// joining kernel, 5.0 TB/s. One of 778 keys: 8.1 us, both launches' latency.
// (Times in this file: captured calls one after the other, over three sets of
// inputs in turn.)
// ---------------------------------------------------------------------------

template <int D, int kWaves, bool kBf16>
__global__ __launch_bounds__(64 * kWaves) void kv8_decode_kernel(Kv8Cache c, const uint16_t* __restrict__ q,
                                                                 int64_t q_stride, uint16_t* __restrict__ out,
                                                                 Parts parts, int group, int splits,
                                                                 float scale_log2) {
  constexpr int kKs = D / 32, kDt = D / 16;  // k-steps of a score, 16-dimension tiles of the output
  __shared__ float so[kWaves][16][D + 4];
  __shared__ float sm[kWaves][16], sl[kWaves][16];

  // splits come last: those that find no keys (wide tables, short sequences)
  // follow those that do, instead of taking the turns of some XCDs, and only
  // say so (16 sequences of 500 keys, tables for 32768: 11.7 us, with splits
  // first more than twice that)
  const int head = static_cast<int>(blockIdx.x) % c.kv_heads, rt = static_cast<int>(blockIdx.x) / c.kv_heads;
  const int b = static_cast<int>(blockIdx.y), split = static_cast<int>(blockIdx.z);
  const Seq seq = sequence(c, b);
  const int rows = seq.n * group;
  if (16 * rt >= rows) return;  // uniform: the whole workgroup leaves
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, h = lane >> 4;
  const int heads = c.kv_heads * group;

  // This lane's query row: token tq of the sequence, head g of the group.
  const int r = 16 * rt + i;
  const bool live = r < rows;
  const int tq = live ? r / group : 0, g = live ? r - tq * group : 0;
  const int limit = live ? min(seq.len - seq.n + tq, seq.seen - 1) : -1;  // last key the row sees
  const uint16_t* const qrow = q + static_cast<int64_t>(seq.row0 + tq) * q_stride + (head * group + g) * D;
  f16x8 qf[kKs];
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live) v = *reinterpret_cast<const u32x4*>(qrow + 64 * (ks / 2) + 16 * h + 8 * (ks % 2));
    qf[ks] = __builtin_bit_cast(f16x8, v);
  }

  // Keys that some row of this tile sees, in tiles of 64, and this split's.
  const int last_t = min(16 * rt + 15, rows - 1) / group;
  const int top = min(seq.len - seq.n + last_t, seq.seen - 1);  // the row tile's last key
  const Span span = tiles_of(top < 0 ? 0 : top / 64 + 1, splits, split, 4);
  const size_t all_rows = static_cast<size_t>(c.tokens) * heads;
  if (splits > 1 && span.first >= span.end) {  // no keys: sums of zero, whose outputs nobody reads
    if (threadIdx.x < 16 && live) {
      const size_t to = static_cast<size_t>(seq.row0 + tq) * heads + head * group + g;
      *reinterpret_cast<f32x2*>(parts.ml + 2 * (split * all_rows + to)) = f32x2{kNegInf, 0.f};
    }
    return;
  }
  const int32_t* const table = c.table + static_cast<size_t>(b) * c.table_width;

  f32x4 o[kDt];
#pragma unroll
  for (int d = 0; d < kDt; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNegInf, l = 0.f;

  // Lane (i, h) reads K rows of the 16 tokens with i / 4 and V of those with h;
  // 16 tokens lie within one page. Where there is no page (behind the last
  // key, or its number is not one of the pool's) page 0 is read and counts for
  // nothing. Page numbers are requested a tile before the codes they lead to.
  auto page_id = [&](int tile, int part) {
    const int t = 64 * tile + 16 * part;
    return tile < span.end && t <= top ? table[t >> c.page_shift] : -1;
  };
  auto known = [&](int id) { return id >= 0 && id < c.num_pages; };
  auto load_k = [&](int tile, int id, u32x4 (&kc)[4][kKs / 2]) {
    const int at = ((64 * tile + 16 * (i >> 2)) & (c.page - 1)) + (i & 3);
    const uint8_t* const base =
        c.k + ((static_cast<size_t>(known(id) ? id : 0) * c.kv_heads + head) * c.page + at) * D + 16 * h;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < kKs / 2; ++x)
        kc[j][x] = *reinterpret_cast<const u32x4*>(base + 4 * j * D + 64 * x);
  };
  auto load_v = [&](int tile, int id, u32x4 (&vc)[kDt]) {
    const int at = (64 * tile + 16 * h) & (c.page - 1);
    const uint8_t* const base =
        c.v + ((static_cast<size_t>(known(id) ? id : 0) * c.kv_heads + head) * D + i) * c.page + at;
#pragma unroll
    for (int d = 0; d < kDt; ++d) vc[d] = *reinterpret_cast<const u32x4*>(base + static_cast<size_t>(16 * d) * c.page);
  };

  u32x4 kc[4][kKs / 2], vc[kDt];
  int tile = span.first + wave;
  int kid = page_id(tile, i >> 2), vid = page_id(tile, h);            // this tile's pages
  int kid1 = page_id(tile + kWaves, i >> 2), vid1 = page_id(tile + kWaves, h);  // and the next one's
  float ksc = 0.f, vsc = 1.f;
  if (tile < span.end) {
    load_k(tile, kid, kc);
    const size_t unit = static_cast<size_t>(known(vid) ? vid : 0) * c.kv_heads + head;
    ksc = c.k_scales[unit];
    vsc = c.v_scales[unit];
    load_v(tile, vid, vc);
  }
  for (; tile < span.end; tile += kWaves) {
    const int kid2 = page_id(tile + 2 * kWaves, i >> 2), vid2 = page_id(tile + 2 * kWaves, h);
    f32x4 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        const u32x4 w = kc[j][ks / 2];
        const f16x8 kf = ks % 2 ? widen<kBf16>(w[2], w[3]) : widen<kBf16>(w[0], w[1]);
        s[j] = mfma_16x16x32<kBf16>(kf, qf[ks], s[j]);
      }
    }
    const bool more = tile + kWaves < span.end;
    if (more) load_k(tile + kWaves, kid1, kc);
    const float f = ksc * scale_log2, lv = log_scale(vsc), iv = 1.f / held_scale(vsc);
    float nks = 0.f, nvs = 1.f;
    if (more) {
      const size_t unit = static_cast<size_t>(known(vid1) ? vid1 : 0) * c.kv_heads + head;
      nks = c.k_scales[unit];
      nvs = c.v_scales[unit];
    }

    // Tokens 64 tile + 16 h + 4 j + e of this lane: seen up to `limit`.
    const int t0 = 64 * tile + 16 * h;
    const int see = known(vid) ? limit - t0 : -1;
    float x[16];
    float mt = kNegInf;
    if (__any(see < 15)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = e <= see ? fmaf(s[e / 4][e % 4], f, lv) : kNegInf;
        mt = fmaxf(mt, x[e]);
      }
      const int count = known(vid) ? top - t0 + 1 : 0;
#pragma unroll
      for (int d = 0; d < kDt; ++d) vc[d] = first_bytes(vc[d], count);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = fmaf(s[e / 4][e % 4], f, lv);
        mt = fmaxf(mt, x[e]);
      }
    }
    mt = fmaxf(mt, __shfl_xor(mt, 16, kWave));
    mt = fmaxf(mt, __shfl_xor(mt, 32, kWave));
    const float mn = fmaxf(m, mt);
    const float ref = mn == kNegInf ? 0.f : mn;
    const float shrink = __builtin_amdgcn_exp2f(m - ref);  // 0 for the first keys
    const float base = ref - kRaise;
    m = mn;
    f32x8 w[2];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float p = __builtin_amdgcn_exp2f(x[e] - base);
      w[e / 8][e % 8] = p;
      sum += p;
    }
    l = fmaf(sum * kLower, iv, l * shrink);
    const f16x8 p0 = to_f16(w[0]), p1 = to_f16(w[1]);
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] *= shrink;
      o[d] = mfma_16x16x32<false>(widen<false>(vc[d][0], vc[d][1]), p0, o[d]);
      o[d] = mfma_16x16x32<false>(widen<false>(vc[d][2], vc[d][3]), p1, o[d]);
    }
    if (more) load_v(tile + kWaves, vid1, vc);
    vid = vid1;
    kid1 = kid2;
    vid1 = vid2;
    ksc = nks;
    vsc = nvs;
  }
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);

  // The wavefronts' parts meet in LDS; lane (i, h) holds dimensions
  // 16 d + 4 h .. + 3 of row i.
#pragma unroll
  for (int d = 0; d < kDt; ++d) *reinterpret_cast<f32x4*>(&so[wave][i][16 * d + 4 * h]) = o[d];
  if (h == 0) {
    sm[wave][i] = m;
    sl[wave][i] = l;
  }
  __syncthreads();
  for (int at = threadIdx.x; at < 16 * (D / 4); at += 64 * kWaves) {
    const int rr = at / (D / 4), d = 4 * (at % (D / 4));
    const int row = 16 * rt + rr;
    if (row >= rows) continue;
    float mx = sm[0][rr];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mx = fmaxf(mx, sm[w][rr]);
    const float base = mx == kNegInf ? 0.f : mx;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][rr] - base);
      total = fmaf(sl[w][rr], f, total);
      const f32x4 part = *reinterpret_cast<const f32x4*>(&so[w][rr][d]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(part[e], f * kLower, v[e]);
    }
    const int t = row / group, gg = row - t * group;
    const size_t to = static_cast<size_t>(seq.row0 + t) * heads + head * group + gg;
    if (splits == 1) {
      const float inv = total == 0.f ? 0.f : 1.f / total;  // (a NaN stays one)
      const uint32_t lo = half_bits<kBf16>(v[0] * inv) | (static_cast<uint32_t>(half_bits<kBf16>(v[1] * inv)) << 16);
      const uint32_t hi = half_bits<kBf16>(v[2] * inv) | (static_cast<uint32_t>(half_bits<kBf16>(v[3] * inv)) << 16);
      *reinterpret_cast<u32x2*>(out + to * D + d) = u32x2{lo, hi};
    } else {
      float* const p = parts.o + (static_cast<size_t>(split) * all_rows + to) * D + d;
      *reinterpret_cast<f32x4*>(p) = v;
      if (d == 0) *reinterpret_cast<f32x2*>(parts.ml + 2 * (static_cast<size_t>(split) * all_rows + to)) = f32x2{mx, total};
    }
  }
}

// ---------------------------------------------------------------------------
// Joins the splits of every row, at most 64: weights 2^(m_z - m), the same
// order every time. Rows of no sequence are left alone. One wavefront takes one
// row; lane z forms the weight of split z, half the lanes then add the outputs
// of even splits, half those of odd ones, eight loads at a time.
// ---------------------------------------------------------------------------

constexpr int kMaxSplits = 64;

template <int D, bool kBf16>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8Cache c, uint16_t* __restrict__ out, Parts parts, int heads,
                                                       int splits) {
  const size_t rows = static_cast<size_t>(c.tokens) * heads;
  const size_t row = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int token = static_cast<int>(row / heads);
  if (token < c.cu[0] || token >= c.cu[c.batch]) return;
  const int lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
  constexpr int kE = D / 32;  // dimensions per lane
  typedef float part __attribute__((ext_vector_type(kE)));
  f32x2 ml = {kNegInf, 0.f};
  if (lane < splits) ml = *reinterpret_cast<const f32x2*>(parts.ml + 2 * (lane * rows + row));
  const float m = wave_max(ml[0]);
  // a split without keys for this row (sum 0) counts for nothing: -1. Every other
  // one is read whatever its weight, so that a NaN reaches the output (0 NaN = NaN).
  const float f = ml[1] == 0.f ? -1.f : __builtin_amdgcn_exp2f(ml[0] - (m == kNegInf ? 0.f : m));
  float total = f < 0.f ? 0.f : ml[1] * f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d, kWave);
  part v = {};
  for (int z0 = 0; z0 < splits; z0 += 16) {  // (the same steps in both halves: weights come from any lane)
    part p[8];
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int z = z0 + 2 * u + h;
      const float weight = __shfl(f, z & 63, kWave);
      w[u] = z < splits ? weight : -1.f;
      p[u] = part{};
      if (w[u] >= 0.f) p[u] = *reinterpret_cast<const part*>(parts.o + (z * rows + row) * D + kE * i);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] = fmaf(p[u][e], w[u], v[e]);
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int e = 0; e < kE; ++e) v[e] = (v[e] + __shfl_xor(v[e], 32, kWave)) * inv;
  if (h != 0) return;
  uint32_t* const to = reinterpret_cast<uint32_t*>(out + row * D + kE * i);
#pragma unroll
  for (int e = 0; e < kE; e += 2) to[e / 2] = half_bits<kBf16>(v[e]) | (static_cast<uint32_t>(half_bits<kBf16>(v[e + 1])) << 16);
}

// ---------------------------------------------------------------------------
// Prompts: a workgroup of eight wavefronts takes 256 rows of one kv head (the
// query heads of the group side by side, so that one K/V tile serves all of
// them) and walks the keys in tiles of 64; each wavefront has 32 rows.
//
// v_mfma_32x32x16: lane (i = lane % 32, h = lane / 32). Row i of a K tile is
// the key with bits 2 and 3 of i exchanged: lane (i, h) then holds, for row i
// of Q, in registers 8 u .. 8 u + 7 the scores of the consecutive keys
// 16 u + 8 h .. + 7, the B operand of the second product, and a register's page
// is the same in every lane.
//
// Per tile and wavefront 1024 cycles of matrix unit (D = 128) face some 230
// vector operations, 32 of them exponentials of four times the cost, and 32
// fragments of 16 bytes per lane from LDS, whose bandwidth is another 1024. So
// - codes are widened once per workgroup on their way into LDS: 16 conversions
//   per wavefront and tile,
// - pages and scales come 16 tiles at a time, one part of 16 keys per lane, and
//   are handed out by v_readlane (scalar loads in every softmax phase, that
//   each phase had to wait for, took 11% longer),
// - the reference of the exponentials follows the maximum lazily: it moves (and
//   the sums are rescaled) only when a score passes it by more than 2^4, so
//   nearly every tile goes without rescaling. Weights are raised by 2^11: at
//   most 2^15, the largest of a row at least 2^11.
//
// The two wavefronts of a SIMD take turns: wavefronts 0-3 and 4-7 (one of each
// per SIMD) walk the same tiles half a step apart, one half in its product
// phase (second product of tile t - 1, scores of tile t) while the other is in
// its softmax phase. Every phase ends at a barrier. What product phase t reads,
// K of tile t and V of tile t - 1 ("pair t"), is one of two buffers: phase t of
// the first half falls on step 2 t, of the second on 2 t + 1, so the other
// buffer is free on both, and each half fills its share of it in its product
// phase, between the MFMAs, from registers loaded a step earlier.
//
// Two sequences of about 4096 and 3000 new tokens over 2048, 32 query heads on
// 8, D = 128: 443 us, 0.88 PFLOP/s; the matrix unit is busy 37% of the time, the
// clock at 2.1 GHz. In copies that skip the rest of the work the products and the
// fills take 369 us, the softmax and the fills 250: the turns hide some two thirds
// of the softmax behind the products.
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr float kLazy = 4.f, kLazyRaise = kRaise - kLazy, kLazyLower = 0x1p-11f;

// The larger of x in lanes l and l ^ 32, in both: the swap leaves the lower
// half's values in one register and the upper half's in the other. (Written
// out: the compiler drops the second result of the builtin.)
__device__ __forceinline__ float halves_max(float x) {
  float lower = x, upper = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(lower), "+v"(upper));
  return fmaxf(lower, upper);
}

constexpr int kPromptRows = 256;  // rows of a row tile

// The n-th row tile of the call: its sequence (-1: there are fewer) and its
// number within it. Every wavefront counts the sequences' tiles, 64 sequences
// at a time, so that the workgroups that have work are the first of the grid:
// a grid of equal parts for every sequence left half of the CUs without any
// while the other half worked (two sequences of 4096 and some 3000 tokens took
// a fifth longer). Workgroups go to the shader engines in strict turn,
// those that end at once took the turns of some.
struct RowTile {
  int b, rt;
};
__device__ __forceinline__ RowTile row_tile(const Kv8Cache& c, int group, int n) {
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < c.batch; b0 += 64) {
    const int tiles = b0 + lane < c.batch ? (sequence(c, b0 + lane).n * group + kPromptRows - 1) / kPromptRows : 0;
    int sum = tiles;  // of this sequence and those before it
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int below = __shfl_up(sum, d, kWave);
      sum += lane >= d ? below : 0;
    }
    const uint64_t behind = __ballot(sum > n);
    if (behind) {
      const int at = __builtin_ctzll(behind);
      return {b0 + at, __builtin_amdgcn_readlane(sum, at) - 1 - n};  // the last tile first
    }
    n -= __builtin_amdgcn_readlane(sum, 63);
  }
  return {-1, 0};
}

template <int D, bool kBf16>
__global__ __launch_bounds__(512) void kv8_prompt_kernel(Kv8Cache c, const uint16_t* __restrict__ q, int64_t q_stride,
                                                         uint16_t* __restrict__ out, Parts parts, int group,
                                                         int splits, float scale_log2) {
  constexpr int kRows = kPromptRows, kKs = D / 16, kDt = D / 32;
  constexpr int kKRow = 2 * D;  // bytes of a widened K row
  constexpr int kKBytes = 64 * kKRow, kVBytes = D * 128;
  constexpr int kBuf = kKBytes + kVBytes;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kBuf];
  lds_u8* const lds = (lds_u8*)(smem);

  // Heads next to each other (the XCDs take workgroups in turn: one that gets
  // the same head again finds its codes in L2), then sequence by sequence the
  // row tiles from the last, whose rows see the most keys, down to the first,
  // so that short workgroups fill the gaps at the end.
  unsigned at = blockIdx.y * gridDim.x + blockIdx.x;
  const int head = static_cast<int>(at % c.kv_heads);
  at /= c.kv_heads;
  const int split = static_cast<int>(at % splits);  // (few: prompts that need splits have few row tiles)
  const RowTile tile = row_tile(c, group, static_cast<int>(at / splits));
  if (tile.b < 0) return;
  const int b = tile.b, rt = tile.rt;
  const Seq seq = sequence(c, b);
  const int rows = seq.n * group;
  if (kRows * rt >= rows) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave >> 2;
  const int i = lane & 31, h = lane >> 5;
  const int heads = c.kv_heads * group;

  const int r = kRows * rt + 32 * wave + i;
  const bool live = r < rows;
  const int tq = live ? r / group : 0, g = live ? r - tq * group : 0;
  const int limit = live ? min(seq.len - seq.n + tq, seq.seen - 1) : -1;  // last key the row sees
  const uint16_t* const qrow = q + static_cast<int64_t>(seq.row0 + tq) * q_stride + (head * group + g) * D;
  f16x8 qf[kKs];
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live) v = *reinterpret_cast<const u32x4*>(qrow + 16 * ks + 8 * h);
    qf[ks] = __builtin_bit_cast(f16x8, v);
  }

  const int last_t = min(kRows * rt + kRows - 1, rows - 1) / group;
  const int top = __builtin_amdgcn_readfirstlane(min(seq.len - seq.n + last_t, seq.seen - 1));  // the last key
  const Span span = tiles_of(top < 0 ? 0 : top / 64 + 1, splits, split, 2);
  const int first = __builtin_amdgcn_readfirstlane(span.first);
  const int tiles = __builtin_amdgcn_readfirstlane(span.end - span.first);

  f32x16 o[kDt], s[2];
  f16x8 w[4];
#pragma unroll
  for (int d = 0; d < kDt; ++d) o[d] = f32x16{};
#pragma unroll
  for (int p = 0; p < 4; ++p) w[p] = f16x8{};  // tile -1: no weights, and zeros for its V
  float base = kNegInf, l = 0.f;

  if (tiles > 0) {
    // Pages and scales, 64 parts of 16 keys (a batch of 16 tiles) at a time:
    // lane p holds those of part p, v_readlane hands them out. The next
    // batch's pages are requested as a batch begins, their scales six tiles
    // later. Every index is that of some key of the sequence; what lies behind
    // the last key counts for nothing.
    const int32_t* const table = c.table + static_cast<size_t>(b) * c.table_width;
    auto known = [&](int id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(c.num_pages); };
    const uint32_t page_bytes = static_cast<uint32_t>(c.kv_heads) * c.page * D;  // <= 2^24

    // A wavefront's share of pair j: for D = 128, 8 rows of K (part wave / 2 of
    // the tile's four parts of 16 keys) and part wave % 4 of 64 rows of V; for
    // D = 64 the first half brings K, 16 rows per wavefront, the second V.
    constexpr bool kBoth = D == 128;
    const bool does_k = kBoth || half == 0, does_v = kBoth || half == 1;
    const int kpart = kBoth ? wave >> 1 : wave & 3, vpart = wave & 3;
    const int krow = kBoth ? 8 * wave + (lane >> 3) : 16 * (wave & 3) + (lane >> 2), kch = lane % (D / 16);
    const int vrow = (kBoth ? 64 * half : 0) + lane;
    const uint32_t koff = static_cast<uint32_t>((krow & 15) * D + 16 * kch), voff = static_cast<uint32_t>(vrow * c.page);
    const uint8_t* const khead = c.k + static_cast<size_t>(head) * c.page * D;
    const uint8_t* const vhead = c.v + static_cast<size_t>(head) * c.page * D;
    auto batch_pages = [&](int n) {
      const uint32_t t = 64u * static_cast<uint32_t>(first + 16 * n) + 16u * static_cast<uint32_t>(lane);
      return table[min(t, static_cast<uint32_t>(top)) >> c.page_shift];
    };
    auto unit = [&](int id) { return static_cast<size_t>(known(id) ? id : 0) * c.kv_heads + head; };
    int id0, id1;             // pages of this batch and of the next
    uint64_t ok;              // parts whose page is known
    float ks1, vs1;           // scales of the next batch
    float f0, off0, iv0;      // of this one: times scale_log2; V's, as log2 and lowered reciprocal
    auto enter_batch = [&]() {
      id0 = id1;
      ok = __ballot(known(id0));
      // (page 0's, where there is no page: a factor of 0 or NaN would turn a masked
      // score's infinity into NaN)
      const float v = known(id0) ? vs1 : 1.f, f = known(id0) ? ks1 * scale_log2 : 1.f;
      f0 = f < 0x1p-126f ? 0x1p-126f : f;
      off0 = log_scale(v);
      iv0 = __builtin_amdgcn_rcpf(held_scale(v)) * kLazyLower;
    };
    auto lane_float = [](float v, int at) {
      return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), at));
    };

    int held = 0;  // keys of the V part in the registers
    u32x4 kreg, vreg;
    auto fetch = [&](int j, int batch) {
      auto page_of = [&](int t, int part) {  // t: a tile of this batch or the next
        const int at = 4 * (t & 15) + part;
        const int here = __builtin_amdgcn_readlane(id0, at), there = __builtin_amdgcn_readlane(id1, at);
        return t >> 4 == batch ? here : there;
      };
      const int tk = 64 * (first + j) + 16 * kpart, tv = 64 * (first + j - 1) + 16 * vpart;
      if (does_k) {
        const int id = page_of(j, kpart);
        const uint8_t* const p = khead + static_cast<uint64_t>(known(id) ? static_cast<uint32_t>(id) : 0u) * page_bytes +
                                 static_cast<uint32_t>((tk & (c.page - 1)) * D);
        kreg = *reinterpret_cast<const u32x4*>(p + koff);
      }
      if (does_v) {
        const int id = page_of(j > 0 ? j - 1 : 0, vpart);
        const uint8_t* const p = vhead + static_cast<uint64_t>(known(id) ? static_cast<uint32_t>(id) : 0u) * page_bytes +
                                 static_cast<uint32_t>(tv & (c.page - 1));
        vreg = *reinterpret_cast<const u32x4*>(p + voff);
        held = known(id) && j > 0 ? top - tv + 1 : 0;  // (the tile before the first: none)
      }
    };
    // 16-byte chunk positions are XOR-ed by the row, so that a fragment read of
    // 32 rows meets no bank twice: K rows of 256 bytes by 16 rows, of 128 bytes
    // (and V rows) by pairs of rows.
    auto k_chunk = [](int row, int ch) {
      return row * kKRow + 16 * (D == 128 ? ch ^ (row & 15) : ch ^ ((row >> 1) & 7));
    };
    auto v_chunk = [](int row, int ch) { return kKBytes + row * 128 + 16 * (ch ^ ((row >> 1) & 7)); };
    const int kto0 = k_chunk(krow, 2 * kch), kto1 = k_chunk(krow, 2 * kch + 1);
    const int vto0 = v_chunk(vrow, 2 * vpart), vto1 = v_chunk(vrow, 2 * vpart + 1);
    // One of the four steps that bring pair j from the registers to LDS.
    auto stage = [&](int j, int step) {
      lds_u8* const to = lds + (j & 1) * kBuf;
      if (step < 2) {
        if (does_k)
          *(lds_u32x4*)(to + (step == 0 ? kto0 : kto1)) =
              __builtin_bit_cast(u32x4, widen<kBf16>(kreg[2 * step], kreg[2 * step + 1]));
      } else if (does_v) {
        if (step == 2 && held < 16) vreg = first_bytes(vreg, held);
        *(lds_u32x4*)(to + (step == 2 ? vto0 : vto1)) =
            __builtin_bit_cast(u32x4, widen<false>(vreg[2 * step - 4], vreg[2 * step - 3]));
      }
    };
    auto phase_end = [&]() {
      wait_counts<63, 0>();  // LDS only: the codes on their way stay in flight
      bare_barrier();
    };

    const int wave_low = __builtin_amdgcn_readfirstlane(
        min(seq.len - seq.n + min(kRows * rt + 32 * wave, rows - 1) / group, seq.seen - 1));  // first row's last key
    const int wave_whole = kRows * rt + 32 * wave + 31 < rows ? wave_low : -1;  // keys that every lane sees
    const int ktok = (i & 19) | ((i & 4) << 1) | ((i & 8) >> 1);  // bits 2 and 3 exchanged
    int kat[kKs], vat[4];
#pragma unroll
    for (int x = 0; x < kKs; ++x) kat[x] = k_chunk(ktok, 2 * x + h);
#pragma unroll
    for (int p = 0; p < 4; ++p) vat[p] = v_chunk(i, 2 * p + h);

    // A product phase: fragments come from LDS in groups of four, two groups
    // ahead of their MFMAs (the fences hold that order; one read at a time
    // would leave the matrix unit waiting for every one of them).
    constexpr int kV = 4 * kDt, kAll = kV + 2 * kKs;  // fragments of V, of both
    auto products = [&](int j, int batch, auto with_scores) {
      constexpr int kGroups = (with_scores ? kAll : kV) / 4;
      const lds_u8* const src = lds + (j & 1) * kBuf;
      u32x4 f[3][4];
      auto read = [&](int gr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 4 * gr + e;
          f[gr % 3][e] = n < kV ? *(const lds_u32x4*)(src + vat[n / kDt % 4] + (n % kDt) * 32 * 128)
                                : *(const lds_u32x4*)(src + kat[(n - kV) / 2 % kKs] + ((n - kV) & 1) * 32 * kKRow);
        }
      };
      if constexpr (with_scores) {
        s[0] = f32x16{};
        s[1] = f32x16{};
      }
      read(0);
      read(1);
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        if (gr + 2 < kGroups) read(gr + 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 4 * gr + e;
          const f16x8 x = __builtin_bit_cast(f16x8, f[gr % 3][e]);
          if (n < kV) {
            o[n % kDt] = mfma_32x32x16<false>(x, w[n / kDt % 4], o[n % kDt]);
          } else {
            s[(n - kV) & 1] = mfma_32x32x16<kBf16>(x, qf[(n - kV) / 2 % kKs], s[(n - kV) & 1]);
          }
          if (with_scores && gr == 1) {
            __builtin_amdgcn_sched_barrier(0);
            stage(j + 1, e);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (with_scores && gr == 2) fetch(j + 2, batch);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    auto softmax = [&](int j) {
      const int t0 = 64 * (first + j);
      const int part = 4 * (j & 15);
      const int seen = static_cast<int>(ok >> part) & 15;
      float f[4], off[4], iv[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        f[p] = lane_float(f0, part + p);
        off[p] = lane_float(off0, part + p);
        iv[p] = lane_float(iv0, part + p);
      }
      if (seen != 15 || t0 + 63 > wave_whole) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int p = 2 * a + e / 8;
            s[a][e] = ((seen >> p) & 1) && t0 + 16 * p + 8 * h + e % 8 <= limit ? s[a][e] : kNegInf;
          }
      }
      float mt = kNegInf;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float mp = s[p / 2][8 * (p % 2)];
#pragma unroll
        for (int e = 1; e < 8; ++e) mp = fmaxf(mp, s[p / 2][8 * (p % 2) + e]);
        mt = fmaxf(mt, fmaf(mp, f[p], off[p]));
      }
      mt = halves_max(mt);
      if (__any(mt > base + kLazy)) {
        const float moved = mt > base + kLazy ? mt : base;
        const float shrink = moved == kNegInf ? 1.f : __builtin_amdgcn_exp2f(base - moved);  // 0 for the first keys
        base = moved;
        l *= shrink;
#pragma unroll
        for (int d = 0; d < kDt; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][e] *= shrink;
      }
      const float ref = (base == kNegInf ? 0.f : base) - kLazyRaise;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float b0 = off[p] - ref;
        f32x8 x;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __builtin_amdgcn_exp2f(fmaf(s[p / 2][8 * (p % 2) + e], f[p], b0));
          sum += x[e];
        }
        l = fmaf(sum, iv[p], l);
        w[p] = to_f16(x);
      }
    };

    id1 = batch_pages(0);
    ks1 = c.k_scales[unit(id1)];
    vs1 = c.v_scales[unit(id1)];
    enter_batch();
    fetch(0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) stage(0, e);
    fetch(1, 0);
    phase_end();
    if (half == 1) phase_end();  // the second half is a step behind
    for (int j = 0; j < tiles; ++j) {
      const int batch = j >> 4;
      if ((j & 15) == 0) {
        if (j > 0) enter_batch();
        id1 = batch_pages(batch + 1);
      }
      if ((j & 15) == 6) {
        ks1 = c.k_scales[unit(id1)];
        vs1 = c.v_scales[unit(id1)];
      }
      __builtin_amdgcn_s_setprio(1);  // its MFMAs go before the other half's vector work
      products(j, batch, std::true_type{});
      __builtin_amdgcn_s_setprio(0);
      phase_end();
      softmax(j);
      phase_end();
    }
    products(tiles, 0, std::false_type{});
    if (half == 0) phase_end();  // the second half's last softmax phase
  }

  l += __shfl_xor(l, 32, kWave);
  if (!live) return;
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] *= kLazyLower;
  const size_t to = static_cast<size_t>(seq.row0 + tq) * heads + head * group + g;
  if (splits == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t b4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) b4[x] = half_bits<kBf16>(o[d][4 * e + x] * inv);
        *reinterpret_cast<u32x2*>(out + to * D + 32 * d + 8 * e + 4 * h) = u32x2{b4[0] | (b4[1] << 16), b4[2] | (b4[3] << 16)};
      }
  } else {
    const size_t at = static_cast<size_t>(split) * c.tokens * heads + to;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(parts.o + at * D + 32 * d + 8 * e + 4 * h) =
            f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
    if (h == 0) *reinterpret_cast<f32x2*>(parts.ml + 2 * at) = f32x2{base, l};
  }
}

// The decode form takes calls of few rows per kv head, and small prompts: a
// prompt workgroup walks its keys one tile after the other, some 2 us each, and
// a small call has few of them. Measured (one sequence, 32 query heads on 8 of
// 128) against row tiles of 16 times kv heads times tiles of 64 keys: 3800 (160
// new tokens over 574) 13.9 us, as a prompt 21.6; 9200 (512 alone) 17.3, 29.9;
// 12600 (300 over 1000) 29.1, 28.5; 31000 (700 over 700) 48.0, 47.9; 35000 (1024
// alone) 41.4, 47.8; 41000 (512 over 2000) 74.6, 45.0. Up to 64 rows it reads the keys hardly more often than the
// prompt form, whatever their number.
constexpr int kDecodeRows = 64;
constexpr int64_t kDecodeTiles = 24576;

template <int D, bool kBf16>
hipError_t launch_dim(const Kv8Cache& c, const uint16_t* q, int64_t q_stride, uint16_t* out, int q_heads, float scale,
                      const Kv8Plan& plan, void* workspace, hipStream_t stream) {
  const int group = q_heads / c.kv_heads;
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int64_t rows = static_cast<int64_t>(most) * group, all = static_cast<int64_t>(c.tokens) * q_heads;
  const float scale_log2 = scale * kLog2e;
  Parts parts = {nullptr, nullptr};
  if (plan.splits > 1) {
    parts.o = static_cast<float*>(workspace);
    parts.ml = parts.o + plan.splits * all * D;
  }
  hipError_t e;
  if (plan.decode) {
    const int row_tiles = static_cast<int>((rows + 15) / 16);
    const dim3 grid(static_cast<uint32_t>(c.kv_heads * row_tiles), static_cast<uint32_t>(c.batch),
                    static_cast<uint32_t>(plan.splits));
    e = plan.waves == 8 ? launch_kernel(kv8_decode_kernel<D, 8, kBf16>, grid, dim3(512), 0, stream, c, q, q_stride, out,
                                        parts, group, plan.splits, scale_log2)
                        : launch_kernel(kv8_decode_kernel<D, 4, kBf16>, grid, dim3(256), 0, stream, c, q, q_stride, out,
                                        parts, group, plan.splits, scale_log2);
  } else {
    constexpr int64_t kWide = int64_t{1} << 22;  // a dimension of the grid stays under 2^32 work-items
    const dim3 grid(static_cast<uint32_t>(plan.prompt_blocks < kWide ? plan.prompt_blocks : kWide),
                    static_cast<uint32_t>((plan.prompt_blocks + kWide - 1) / kWide));
    e = launch_kernel(kv8_prompt_kernel<D, kBf16>, grid, dim3(512), 0, stream, c, q, q_stride, out, parts, group,
                      plan.splits, scale_log2);
  }
  if (e != hipSuccess || plan.splits == 1) return e;
  return launch_kernel(kv8_join_kernel<D, kBf16>, dim3(static_cast<uint32_t>((all + 3) / 4)), dim3(256), 0, stream, c,
                       out, parts, q_heads, plan.splits);
}

}  // namespace

// The keys of a sequence are split over workgroups. For prompts until the
// launch holds 256 workgroups (512 new tokens over 2000, 32 query heads on 8:
// 45.0 us; until 128 61.0, until 512 60.8), a split keeping at least two tiles
// of 64 keys of the longest sequence that the tables can hold. For decode (8 kv heads):
// - up to eight tiles stay whole: the joining kernel costs more than it saves
//   (one sequence of 300 keys: 6.7 us, in two splits 8.1; 16 of 500: 8.2, 9.6);
//   with eight wavefronts where CUs are free for them (6.4, 7.7), which also
//   spares up to 16 tiles the splits from 128 workgroups on (16 sequences of 900:
//   11.3 us, split 12.0; 32: 12.7, 16.3; but 8: 10.7, 9.2),
// - until 512 workgroups, at least four tiles each, one per wavefront (one
//   sequence of 777 keys: four splits 8.1 us, two 10.1, one 10.9; 64 of 1000:
//   whole 20.4 us, in two splits 24.9, in four 26.7),
// - until 2048 where 32 tiles are left to each, which evens out sequences of
//   different lengths (64 of up to 8192 keys: four splits 135 us, one 141-146).
// How long the sequences are is known on the GPU only: there each is cut evenly.
Kv8Plan plan_kv8_attention(const Kv8Cache& c, int q_heads) {
  Kv8Plan p;
  const int group = q_heads / c.kv_heads;
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int64_t rows = static_cast<int64_t>(most) * group;
  const int64_t tiles = (static_cast<int64_t>(c.table_width) * c.page + 63) / 64;
  // row tiles of all sequences: no more than if every one left the last of its
  // tiles all but empty
  auto row_tiles = [&](int64_t size) {
    const int64_t even = c.batch * ((rows + size - 1) / size);
    const int64_t bound = (static_cast<int64_t>(c.tokens) * group + (size - 1) * c.batch) / size;
    return even < bound ? even : bound;
  };
  // (what its grid covers counts, the longest sequence's row tiles for every one)
  p.decode = rows <= kDecodeRows || c.batch * ((rows + 15) / 16) * c.kv_heads * tiles <= kDecodeTiles;
  p.waves = p.decode ? 4 : 8;
  const int64_t groups = row_tiles(p.decode ? 16 : kPromptRows) * c.kv_heads;
  auto until = [&](int64_t workgroups, int64_t least) {
    const int64_t fill = groups > 0 ? workgroups / groups : 1, fit = (tiles + least - 1) / least;
    return fill < fit ? fill : fit;
  };
  int64_t splits = until(256, 2);
  if (p.decode) {
    const int64_t few = until(512, 4), many = until(2048, 32);
    splits = tiles <= 8 ? 1 : few > many ? few : many;
    if (groups <= 256 && tiles > 4 && tiles <= (groups >= 128 ? 16 : 8)) {
      p.waves = 8;
      splits = 1;
    }
  }
  if (splits > kMaxSplits) splits = kMaxSplits;
  // the joining kernel takes four rows per workgroup of 256: under 2^32 work-items
  if (static_cast<int64_t>(c.tokens) * q_heads >= (int64_t{1} << 26)) splits = 1;
  p.splits = splits < 1 ? 1 : static_cast<int>(splits);
  p.prompt_blocks = p.decode ? 0 : groups * p.splits;
  p.workspace_bytes =
      p.splits > 1 ? static_cast<size_t>(p.splits) * c.tokens * q_heads * (c.head_dim + 2) * sizeof(float) : 0;
  return p;
}

hipError_t launch_kv8_attention(const Kv8Cache& c, const uint16_t* q, int64_t q_stride, uint16_t* out, int q_heads,
                                float softmax_scale, const Kv8Plan& plan, void* workspace, bool bf16,
                                hipStream_t stream) {
  if (c.head_dim == 128)
    return bf16 ? launch_dim<128, true>(c, q, q_stride, out, q_heads, softmax_scale, plan, workspace, stream)
                : launch_dim<128, false>(c, q, q_stride, out, q_heads, softmax_scale, plan, workspace, stream);
  if (c.head_dim == 64)
    return bf16 ? launch_dim<64, true>(c, q, q_stride, out, q_heads, softmax_scale, plan, workspace, stream)
                : launch_dim<64, false>(c, q, q_stride, out, q_heads, softmax_scale, plan, workspace, stream);
  return hipErrorInvalidValue;
}

}  // namespace mq
