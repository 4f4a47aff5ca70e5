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
//   x_t = score_t log2(e) + log2(v_scale_t),   m = max x_t,   w_t = 2^(x_t - m) <= 1
// the second product is sum w_t code_t in units of 2^m whatever the scales of
// the pages are, and the sum of the weights is sum w_t / v_scale_t. w is
// rounded once, to fp16 (11 bits; bf16 would lose three more and gains
// nothing, as w <= 1).
//
// Keys that a row does not see get the weight 0 by a select, and V codes
// behind the last token are cleared, so whatever a page holds there (NaN codes
// too) counts for nothing; so do pages whose number is not one of the pool's.
// A row that sees no key is 0.
#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace mq {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_inff();
// Scales outside what the append writes would carry sums out of binary32.
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p120f;

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
// in tiles of 16. A workgroup of four wavefronts takes one such tile and a
// range of keys, a wavefront every fourth tile of 64 keys. Bound by the cache
// read: K and V go from memory straight into registers (16-byte loads, whole
// 64-byte pieces of a page row), K of the next tile is requested as soon as
// this tile's scores are formed, V as soon as its product is, and several
// wavefronts per SIMD keep the loads of a compute unit outstanding.
// v_mfma_16x16x32: lane (i = lane % 16, h = lane / 16). Row i of K tile j is
// token 16 (i / 4) + 4 j + i % 4, so lane (i, h) ends up with the scores of
// row i of Q for tokens 16 h .. 16 h + 15, in order.
// ---------------------------------------------------------------------------

template <int D, bool kBf16>
__global__ __launch_bounds__(256) void kv8_decode_kernel(Kv8Cache c, const uint16_t* __restrict__ q, int64_t q_stride,
                                                         uint16_t* __restrict__ out, Parts parts, int group,
                                                         int row_tiles, int splits, float scale_log2) {
  constexpr int kKs = D / 32, kDt = D / 16;  // k-steps of a score, 16-dimension tiles of the output
  __shared__ float so[4][16][D + 4];
  __shared__ float sm[4][16], sl[4][16];

  const int split = static_cast<int>(blockIdx.x) % splits;
  const int head = static_cast<int>(blockIdx.y) % c.kv_heads, rt = static_cast<int>(blockIdx.y) / c.kv_heads;
  const int b = static_cast<int>(blockIdx.z);
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
  int kid1 = page_id(tile + 4, i >> 2), vid1 = page_id(tile + 4, h);  // and the next one's
  float ksc = 0.f, vsc = 1.f;
  if (tile < span.end) {
    load_k(tile, kid, kc);
    const size_t unit = static_cast<size_t>(known(vid) ? vid : 0) * c.kv_heads + head;
    ksc = c.k_scales[unit];
    vsc = c.v_scales[unit];
    load_v(tile, vid, vc);
  }
  for (; tile < span.end; tile += 4) {
    const int kid2 = page_id(tile + 8, i >> 2), vid2 = page_id(tile + 8, h);
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
    const bool more = tile + 4 < span.end;
    if (more) load_k(tile + 4, kid1, kc);
    const float vs = held_scale(vsc);
    const float f = ksc * scale_log2, lv = __builtin_amdgcn_logf(vs), iv = 1.f / vs;
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
    const float base = mn == kNegInf ? 0.f : mn;
    const float shrink = __builtin_amdgcn_exp2f(m - base);  // 0 for the first keys
    m = mn;
    f32x8 w[2];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float p = __builtin_amdgcn_exp2f(x[e] - base);
      w[e / 8][e % 8] = p;
      sum += p;
    }
    l = fmaf(sum, iv, l * shrink);
    const f16x8 p0 = to_f16(w[0]), p1 = to_f16(w[1]);
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] *= shrink;
      o[d] = mfma_16x16x32<false>(widen<false>(vc[d][0], vc[d][1]), p0, o[d]);
      o[d] = mfma_16x16x32<false>(widen<false>(vc[d][2], vc[d][3]), p1, o[d]);
    }
    if (more) load_v(tile + 4, vid1, vc);
    vid = vid1;
    kid1 = kid2;
    vid1 = vid2;
    ksc = nks;
    vsc = nvs;
  }
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);

  // The four wavefronts' parts meet in LDS; lane (i, h) holds dimensions
  // 16 d + 4 h .. + 3 of row i.
#pragma unroll
  for (int d = 0; d < kDt; ++d) *reinterpret_cast<f32x4*>(&so[wave][i][16 * d + 4 * h]) = o[d];
  if (h == 0) {
    sm[wave][i] = m;
    sl[wave][i] = l;
  }
  __syncthreads();
  const size_t all_rows = static_cast<size_t>(c.tokens) * heads;
  for (int at = threadIdx.x; at < 16 * (D / 4); at += 256) {
    const int rr = at / (D / 4), d = 4 * (at % (D / 4));
    const int row = 16 * rt + rr;
    if (row >= rows) continue;
    const float mx = fmaxf(fmaxf(sm[0][rr], sm[1][rr]), fmaxf(sm[2][rr], sm[3][rr]));
    const float base = mx == kNegInf ? 0.f : mx;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][rr] - base);
      total = fmaf(sl[w][rr], f, total);
      const f32x4 part = *reinterpret_cast<const f32x4*>(&so[w][rr][d]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(part[e], f, v[e]);
    }
    const int t = row / group, gg = row - t * group;
    const size_t to = static_cast<size_t>(seq.row0 + t) * heads + head * group + gg;
    if (splits == 1) {
      const float inv = total > 0.f ? 1.f / total : 0.f;
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
// Joins the splits of every row: weights 2^(m_z - m), in split order. Rows of
// no sequence are left alone. One wavefront takes one row.
// ---------------------------------------------------------------------------

template <int D, bool kBf16>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8Cache c, uint16_t* __restrict__ out, Parts parts, int heads,
                                                       int splits) {
  const size_t rows = static_cast<size_t>(c.tokens) * heads;
  const size_t row = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int token = static_cast<int>(row / heads);
  if (token < c.cu[0] || token >= c.cu[c.batch]) return;
  const int lane = threadIdx.x & 63;
  constexpr int kE = D / 64;
  float m = kNegInf;
  for (int z = lane; z < splits; z += 64) m = fmaxf(m, parts.ml[2 * (z * rows + row)]);
  m = wave_max(m);
  const float base = m == kNegInf ? 0.f : m;
  float total = 0.f, v[kE] = {};
  for (int z = 0; z < splits; ++z) {
    const f32x2 ml = *reinterpret_cast<const f32x2*>(parts.ml + 2 * (z * rows + row));
    if (!(ml[1] > 0.f)) continue;  // a split without keys for this row (its output is not read)
    const float f = __builtin_amdgcn_exp2f(ml[0] - base);
    total = fmaf(ml[1], f, total);
    const float* const p = parts.o + (z * rows + row) * D + kE * lane;
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] = fmaf(p[e], f, v[e]);
  }
  const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) out[row * D + kE * lane + e] = half_bits<kBf16>(v[e] * inv);
}

// ---------------------------------------------------------------------------
// Prompts: a workgroup of eight wavefronts takes 256 rows of one kv head (the
// query heads of the group side by side, so that one K/V tile serves all of
// them) and walks the keys in tiles of 64; each wavefront has 32 rows.
//
// v_mfma_32x32x16: lane (i = lane % 32, h = lane / 32). Row i of half a of a K
// tile (32 keys) is the key with the bits (4 3 2) of i turned to (3 2 4): lane
// (i, h) then holds, for row i of Q, in registers 0 .. 15 the scores of the 16
// consecutive keys 32 a + 16 h + 0 .. 15. They lie in one page, so the scales
// are lane values, and the first and second eight are, widened to fp16, the B
// operands of two steps of the second product, whose A operands are the two
// halves of one 16-byte piece of a V row.
//
// A tile is 1024 cycles of matrix unit per wavefront (D = 128) and as many of
// vector unit (exponentials first of all), so the two wavefronts of a SIMD take
// turns: wavefronts 0-3 and 4-7 (one of each per SIMD) walk the same tiles half
// a step apart, one half in its product phase (second product of tile t - 1,
// scores of tile t) while the other is in its softmax phase. Every phase ends
// at a barrier.
//
// Codes move from memory into LDS untouched (DMA, no registers) and are
// widened as a wavefront reads them, under its MFMAs: widening them once per
// workgroup on the way into LDS cost the softmax phase, the longer one, more
// than it saved, and twice the LDS traffic. What product phase t reads, K of
// tile t and V of tile t - 1 ("pair t"), is one of three buffers. Phase t of
// the first half falls on step 2 t, of the second on 2 t + 1; the first half
// requests pair t + 2 in its softmax phase on step 2 t + 1, the second pair
// t + 3 on 2 t + 2, when the buffer's last readers (pair t - 1, pair t) are past
// it, and both wait at the next softmax phase, two steps later, before a
// barrier that precedes the pair's first use.
//
// The reference of the exponentials follows the maximum lazily: it moves (and
// the sums are rescaled) only when a score passes it by more than 2^8, so
// weights stay at most 2^8 and nearly every tile goes without rescaling.
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef const __attribute__((address_space(1))) void gbl_void;

constexpr float kLazy = 8.f;

// The larger of x in lanes l and l ^ 32, in both: the swap leaves the lower
// half's values in one register and the upper half's in the other. (Written
// out: the compiler drops the second result of the builtin.)
__device__ __forceinline__ float halves_max(float x) {
  float lower = x, upper = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(lower), "+v"(upper));
  return fmaxf(lower, upper);
}

template <int D, bool kBf16>
__global__ __launch_bounds__(512) void kv8_prompt_kernel(Kv8Cache c, const uint16_t* __restrict__ q, int64_t q_stride,
                                                         uint16_t* __restrict__ out, Parts parts, int group,
                                                         int row_tiles, int splits, float scale_log2) {
  constexpr int kRows = 256, kKk = D / 32, kDt = D / 32;  // 16-byte steps of a K row per lane; 32-row tiles of V
  constexpr int kBytes = 64 * D;                          // of K, and of V, in a tile
  constexpr int kSlots = 3;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kSlots * 2 * kBytes];
  lds_u8* const lds = (lds_u8*)(smem);

  // the last rows of a sequence see the most keys: they go first
  const int rt = row_tiles - 1 - static_cast<int>(blockIdx.x) / splits, split = static_cast<int>(blockIdx.x) % splits;
  const int head = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
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
  // k-steps 2 kk and 2 kk + 1 are the halves of the 16-byte pieces 2 kk + h of the K rows
  f16x8 qf[2 * kKk];
#pragma unroll
  for (int ks = 0; ks < 2 * kKk; ++ks) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live) v = *reinterpret_cast<const u32x4*>(qrow + 32 * (ks / 2) + 16 * h + 8 * (ks % 2));
    qf[ks] = __builtin_bit_cast(f16x8, v);
  }

  const int last_t = min(kRows * rt + kRows - 1, rows - 1) / group;
  const int top = min(seq.len - seq.n + last_t, seq.seen - 1);  // the workgroup's last key
  const Span span = tiles_of(top < 0 ? 0 : top / 64 + 1, splits, split, 8);
  const int tiles = span.end - span.first;

  f32x16 o[kDt], s[2];
  f16x8 w[4];
#pragma unroll
  for (int d = 0; d < kDt; ++d) o[d] = f32x16{};
#pragma unroll
  for (int p = 0; p < 4; ++p) w[p] = f16x8{};
  float base = kNegInf, l = 0.f;

  if (tiles > 0) {
    const int32_t* const table = c.table + static_cast<size_t>(b) * c.table_width;
    // Every lane's page numbers and addresses are those of some key of the
    // sequence, so that all loads go out without branches; what lies outside
    // the split or behind the last key is never used or counts for nothing.
    auto page_at = [&](int t) { return table[min(max(t, 0), top) >> c.page_shift]; };
    auto known = [&](int id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(c.num_pages); };
    const uint32_t page_bytes = static_cast<uint32_t>(c.kv_heads) * c.page * D;  // <= 2^24

    // DMA: a wavefront's load fills 1 KB of LDS, lane L the piece at 16 L. K
    // rows are D bytes, V rows 64 (keys); the 16-byte pieces of a row are
    // XOR-ed so that 16 lanes of a fragment read fall on different banks
    // (rows of K in the order above, rows of V consecutive).
    constexpr int kPer = D / 16;  // pieces of a K row
    constexpr int kLoads = kBytes / 1024;  // of K, and of V
    static_assert(kLoads == 8 || kLoads == 4, "one load of both, or of either, per wavefront");
    auto k_piece = [](int row, int piece) {
      return D == 128 ? piece ^ (((row >> 1) & 3) | ((row >> 2) & 4)) : piece ^ (((row >> 2) & 1) | ((row >> 3) & 2));
    };
    auto v_piece = [](int row, int piece) { return piece ^ ((row >> 2) & 3); };
    const bool does_k = kLoads == 8 || half == 0, does_v = kLoads == 8 || half == 1;
    const int wl = wave & (kLoads - 1);
    const int krow = wl * (1024 / D) + lane / kPer, kfrom = 16 * k_piece(krow, lane % kPer);
    const int vrow = wl * 16 + lane / 4, vpart = v_piece(vrow, lane % 4);
    const uint8_t* const kbase = c.k + static_cast<size_t>(head) * c.page * D + kfrom;
    const uint8_t* const vbase = c.v + static_cast<size_t>(head) * c.page * D + vrow * c.page;
    int kid, vid;
    auto request_pages = [&](int j) {
      kid = page_at(64 * (span.first + j) + krow);
      vid = page_at(64 * (span.first + j - 1) + 16 * vpart);
    };
    auto request_pair = [&](int j) {
      const int t = 64 * (span.first + j);
      lds_u8* const to = lds + (j % kSlots) * 2 * kBytes + wl * 1024;
      if (does_k) {
        const uint8_t* const p = kbase + static_cast<uint64_t>(known(kid) ? static_cast<uint32_t>(kid) : 0u) * page_bytes +
                                 ((t + krow) & (c.page - 1)) * D;
        __builtin_amdgcn_global_load_lds((gbl_void*)p, (lds_void*)to, 16, 0, 0);
      }
      if (does_v) {
        const uint8_t* const p = vbase + static_cast<uint64_t>(known(vid) ? static_cast<uint32_t>(vid) : 0u) * page_bytes +
                                 ((t - 64 + 16 * vpart) & (c.page - 1));
        __builtin_amdgcn_global_load_lds((gbl_void*)p, (lds_void*)(to + kBytes), 16, 0, 0);
      }
    };
    // Scales of this lane's 16 keys in each half of a tile, requested a tile
    // ahead, their pages two.
    int sid[2], okid[2];
    float ks[2], vs[2];
    auto request_scale_pages = [&](int j) {
#pragma unroll
      for (int a = 0; a < 2; ++a) sid[a] = page_at(64 * (span.first + j) + 32 * a + 16 * h);
    };
    auto request_scales = [&]() {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        okid[a] = known(sid[a]);
        const size_t unit = static_cast<size_t>(okid[a] ? sid[a] : 0) * c.kv_heads + head;
        ks[a] = c.k_scales[unit];
        vs[a] = c.v_scales[unit];
      }
    };
    auto phase_end = [&]() {
      wait_counts<63, 0>();  // LDS only: what was requested stays in flight
      bare_barrier();
    };

    // Fragment reads: this lane's K row and its piece 2 kk + h, V row and piece 2 p + h.
    const int ktok = ((i & 4) << 2) | ((i >> 1) & 12) | (i & 3);
    int kat[kKk], vat[2];
#pragma unroll
    for (int kk = 0; kk < kKk; ++kk) kat[kk] = ktok * D + 16 * k_piece(ktok, 2 * kk + h);
#pragma unroll
    for (int p = 0; p < 2; ++p) vat[p] = kBytes + i * 64 + 16 * v_piece(i, 2 * p + h);

    int count[2] = {0, 0};  // keys of this lane's V pieces that exist; before the first tile none
    bool ragged = true;     // some lane's are fewer than 16

    // A product phase. Reads go out ahead of the MFMAs that use them; the
    // fences keep them there (one at a time would leave the matrix unit waiting
    // for each).
    auto products = [&](int j, auto with_scores) {
      const lds_u8* const src = lds + (j % kSlots) * 2 * kBytes;
      u32x4 rv[2][kDt], rk[2][kKk];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int d = 0; d < kDt; ++d) rv[p][d] = *(const lds_u32x4*)(src + vat[p] + d * 32 * 64);
      auto read_k = [&](int a) {
        if constexpr (with_scores) {
#pragma unroll
          for (int kk = 0; kk < kKk; ++kk) rk[a][kk] = *(const lds_u32x4*)(src + kat[kk] + a * 32 * D);
        }
      };
      if (ragged) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int d = 0; d < kDt; ++d) rv[p][d] = first_bytes(rv[p][d], count[p]);
      }
      read_k(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int d = 0; d < kDt; ++d) {
          o[d] = mfma_32x32x16<false>(widen<false>(rv[p][d][0], rv[p][d][1]), w[2 * p], o[d]);
          o[d] = mfma_32x32x16<false>(widen<false>(rv[p][d][2], rv[p][d][3]), w[2 * p + 1], o[d]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (p == 0) read_k(1);
      }
      if constexpr (with_scores) {
        s[0] = f32x16{};
        s[1] = f32x16{};
#pragma unroll
        for (int kk = 0; kk < kKk; ++kk)
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            s[a] = mfma_32x32x16<kBf16>(widen<kBf16>(rk[a][kk][0], rk[a][kk][1]), qf[2 * kk], s[a]);
            s[a] = mfma_32x32x16<kBf16>(widen<kBf16>(rk[a][kk][2], rk[a][kk][3]), qf[2 * kk + 1], s[a]);
          }
      }
    };

    auto softmax = [&](int j) {
      const int t0 = 64 * (span.first + j) + 16 * h;
      float f[2], lv[2], iv[2];
      int see[2];
      // Everything that was requested two steps ago has arrived: the pair
      // that the next phases read, the scales, the page numbers.
      wait_counts<0, 15>();
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const float v = held_scale(vs[a]);
        f[a] = fmaxf(ks[a] * scale_log2, 0x1p-126f);  // (0 would turn a masked score's infinity into NaN)
        lv[a] = __builtin_amdgcn_logf(v);
        iv[a] = __builtin_amdgcn_rcpf(v);
        see[a] = okid[a] ? limit - (t0 + 32 * a) : -1;
        count[a] = okid[a] ? top - (t0 + 32 * a) + 1 : 0;
      }
      ragged = __any(min(count[0], count[1]) < 16);
      request_pair(j + 2 + half);
      request_pages(j + 3 + half);
      request_scales();
      request_scale_pages(j + 2);

      if (__any(min(see[0], see[1]) < 15)) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[a][e] = e <= see[a] ? s[a][e] : kNegInf;
      }
      float mt = kNegInf;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float ma = s[a][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) ma = fmaxf(ma, s[a][e]);
        mt = fmaxf(mt, fmaf(ma, f[a], lv[a]));
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
      const float ref = base == kNegInf ? 0.f : base;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const float off = lv[a] - ref;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f32x8 x;
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            x[z] = __builtin_amdgcn_exp2f(fmaf(s[a][8 * e + z], f[a], off));
            sum[e] += x[z];
          }
          w[2 * a + e] = to_f16(x);
          asm volatile("" : "+v"(w[2 * a + e]));  // formed in this phase, not where it is used
        }
        l = fmaf(sum[0] + sum[1], iv[a], l);
      }
    };

    request_pages(0);
    request_pair(0);
    request_pages(1);
    request_pair(1);
    request_pages(2);
    request_scale_pages(0);
    request_scales();
    request_scale_pages(1);
    wait_counts<0, 0>();
    bare_barrier();
    if (half == 1) {  // the second half's first step: it has nothing to compute yet
      request_pair(2);
      request_pages(3);
      phase_end();
    }
    for (int j = 0; j < tiles; ++j) {
      products(j, std::true_type{});
      phase_end();
      softmax(j);
      phase_end();
    }
    products(tiles, std::false_type{});
    if (half == 0) phase_end();  // the second half's last softmax phase
    wait_counts<0, 0>();         // nothing may arrive in LDS after the workgroup has ended
  }

  l += __shfl_xor(l, 32, kWave);
  if (!live) return;
  const size_t to = static_cast<size_t>(seq.row0 + tq) * heads + head * group + g;
  if (splits == 1) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
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

constexpr int kDecodeRows = 64;  // rows of one kv head that the decode form takes (four tiles of 16)
constexpr int kMaxSplits = 64;

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
    const dim3 grid(static_cast<uint32_t>(plan.splits), static_cast<uint32_t>(c.kv_heads * row_tiles),
                    static_cast<uint32_t>(c.batch));
    e = launch_kernel(kv8_decode_kernel<D, kBf16>, grid, dim3(256), 0, stream, c, q, q_stride, out, parts, group,
                      row_tiles, plan.splits, scale_log2);
  } else {
    const int row_tiles = static_cast<int>((rows + 255) / 256);
    const dim3 grid(static_cast<uint32_t>(row_tiles * plan.splits), static_cast<uint32_t>(c.kv_heads),
                    static_cast<uint32_t>(c.batch));
    e = launch_kernel(kv8_prompt_kernel<D, kBf16>, grid, dim3(512), 0, stream, c, q, q_stride, out, parts, group,
                      row_tiles, plan.splits, scale_log2);
  }
  if (e != hipSuccess || plan.splits == 1) return e;
  return launch_kernel(kv8_join_kernel<D, kBf16>, dim3(static_cast<uint32_t>((all + 3) / 4)), dim3(256), 0, stream, c,
                       out, parts, q_heads, plan.splits);
}

}  // namespace

// The keys of a sequence are split over workgroups until the launch holds
// about kTarget of them; a split keeps at least four tiles of 64 keys (eight
// for prompts), of the longest sequence that the tables can hold. How long
// the sequences are is known on the GPU only: there each is cut evenly.
Kv8Plan plan_kv8_attention(const Kv8Cache& c, int q_heads) {
  Kv8Plan p;
  const int group = q_heads / c.kv_heads;
  const int most = c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
  const int64_t rows = static_cast<int64_t>(most) * group;
  p.decode = rows <= kDecodeRows;
  const int64_t tiles = (static_cast<int64_t>(c.table_width) * c.page + 63) / 64;
  const int64_t groups = static_cast<int64_t>(c.batch) * c.kv_heads * (p.decode ? (rows + 15) / 16 : (rows + 255) / 256);
  const int64_t target = p.decode ? 2048 : 256, least = p.decode ? 4 : 8;
  int64_t splits = groups > 0 ? target / groups : 1;
  const int64_t fit = (tiles + least - 1) / least;
  if (splits > fit) splits = fit;
  if (splits > kMaxSplits) splits = kMaxSplits;
  // the joining kernel takes four rows per workgroup of 256: under 2^32 work-items
  if (static_cast<int64_t>(c.tokens) * q_heads >= (int64_t{1} << 26)) splits = 1;
  p.splits = splits < 1 ? 1 : static_cast<int>(splits);
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
