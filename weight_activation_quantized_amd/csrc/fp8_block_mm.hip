// e4m3 matrix product with one scale per block of 128, for gfx950
// (fp8_block_gemv.hip takes up to 16 tokens that fit LDS).
//
//   y[m,n] = rne16( sum_b (sx[b,m] * sw[n/128,b]) * sum_{k in block b} xq[m,k] * wq[n,k] )
//
// with b the blocks of 128 along K, the sums and the scale product in
// binary32. Inside the fp8 matrix unit the products of 8 consecutive k are
// aligned to the largest exponent among them and cut off 2^-13 below it
// (measured, the same on every fp8 form); the groups' sums are binary32. That
// is the price of the fp8 rate: at most 7 * 2^-13 of a group's largest
// product, about 1e-5 of a typical result, far below the output's rounding.
//
// Design:
// - v_mfma_f32_32x32x64_f8f6f4: the fp8 form with twice the rate of the
//   32x32x16 one. Two of them cover one block of 128; their sum starts from
//   zero for every block and is then added to the running sum with one fused
//   multiply-add per value by the block's scale. That is 16 VALU operations
//   (64 cycles) for 128 cycles of matrix unit, so a wavefront takes whole
//   blocks (a split of a block's K over wavefronts would double the VALU work
//   to parity with the MFMAs), and each SIMD has two wavefronts or more so
//   that one's multiply-adds run under another's MFMAs.
// - Weight rows are the MFMA's A operand and token rows its B operand: a lane
//   of the 32x32 result holds one token, so the scale sx * sw is one value
//   per lane and tile (sw is uniform: a tile of 32 channels lies within one
//   block of 128).
// - Tiles move HBM -> LDS by buffer_load ... lds, one or more stages of 128
//   bytes of K ahead of the compute. LDS rows are 128 bytes, their 16-byte
//   chunks XOR-swizzled by the row, so a fragment read of 32 rows meets no
//   bank conflict. Loads past the buffer's end return zero (ragged M, N, K).
// - A lane's 32 bytes of a k-step are the chunks 4 t + h and 4 t + 2 + h of
//   its row; which k a lane holds does not matter as long as both operands
//   agree (and 8 consecutive k stay together: the groups above).
// - Four tile sizes, and for few tiles ranges of K whose binary32 sums a
//   second kernel adds in order (plan_fp8_block_mm says when).
// - Workgroups go round-robin over the 8 XCDs; each XCD gets a contiguous run
//   of tiles in groups of kGroupM token tiles, so that what a run shares stays
//   in its L2.
//
// What bounds it, at 4096 tokens x 4096 x 24576 (256 x 256 tiles, 407 us, 2.0
// PFLOP/s): the matrix unit is busy 46% of the time. Copies that skip work take
// 351 us without the multiply-adds, 275 without the fills, 285 with the fills and
// the output alone: neither hides behind the other, since all wavefronts meet at
// the barrier that starts a stage and wait there for their first fragments. Two
// halves of the workgroup half a stage apart, one reading while the other
// multiplies, were 7% slower: a single wavefront reads its fragments more slowly
// than the other's MFMAs run. The smaller tiles are bound by their fills: 517
// tokens at 4096 x 6144 (64 x 128 tiles) take 26.4 us, without the fills 16.0,
// with the fills and the output alone 24.2; 48 at 12288 x 4096 with the joining
// kernel 15.0, 6.9 and 13.3. The next stage's fragments read before the barrier
// changed nothing there.
//
// Times in this file: captured calls one after the other, over three sets of
// inputs in turn.
#include "block8_launch.h"
#include "device_common.h"

namespace mq {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int kBK = 128;                  // bytes of K per stage: one scale block
constexpr int kGroupM = 4;                // token tiles per group in the tile order
constexpr uint32_t kOob = 0x80000000u;    // a buffer offset past every tile: the load returns 0
constexpr int kBufferFlags = 0x00020000;  // gfx9 buffer descriptor word 3 (raw 32-bit data)

__device__ __forceinline__ int chunk_swizzle(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, kBufferFlags);
}

// A workgroup computes BM tokens x BN channels over a range of stages; its
// WM x WN wavefronts stand over the tile, each with 32 TB tokens x 32 TA
// channels. SLOTS stages of LDS: SLOTS - 1 are in flight or waiting while one
// is computed.
template <int BM_, int BN_, int WM_, int WN_, int SLOTS_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kSlots = SLOTS_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int TB = BM / WM / 32, TA = BN / WN / 32;
  static constexpr int kTiles = (BM + BN) * kBK;               // bytes of the operands in a stage
  static constexpr int kStage = kTiles + 4 * BM + 256;         // behind them scales: of the tokens, of the channel blocks
  static constexpr int kPitch = BN * 2 + 16;  // staged output rows
  static constexpr int kLds = kSlots * kStage > BM * kPitch ? kSlots * kStage : BM * kPitch;
  static constexpr int kLoadsX = BM / 8 / kWaves;              // fills per wavefront and stage (8 rows of 128 bytes each)
  static constexpr int kLoadsT = kLoadsX + BN / 8 / kWaves;
  static constexpr int kLoads = kLoadsT + 1;                   // the last one: scales
  static constexpr int kAhead = (kSlots - 2) * kLoads;         // fills that may be in flight at a round's end
  static_assert(kLds <= 160 * 1024, "LDS capacity");
  static_assert(TA >= 1 && TB >= 1 && BM == 32 * TB * WM && BN == 32 * TA * WN, "wavefront tiles");
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "a wavefront's fills do not straddle the operands");
  static_assert(128 % BN == 0 || BN % 128 == 0, "a tile of 32 channels lies in one scale block");
  static_assert(kAhead < 63, "vmcnt range");
  static_assert(BM % 64 == 0 && kWaves > BM / 64, "a wavefront for every 64 tokens' scales and one for the channels'");
  static_assert(128 % (32 * TA) == 0, "the channels of a wavefront lie in one block");
};

// kSplit: the stages of a tile are cut into `splits` contiguous ranges of
// `share`, one workgroup each, whose binary32 sums go to part[split][M][N].
template <typename S, bool kSplit, bool kBf16>
__global__ __launch_bounds__(S::kThreads) void fp8_block_mm_kernel(
    const uint8_t* __restrict__ xq, const float* __restrict__ s_x, const uint8_t* __restrict__ wq,
    const float* __restrict__ s_w, uint16_t* __restrict__ y, float* __restrict__ part, int M, int N, int K,
    int tiles_m, int tiles_n, int per_xcd, int splits, int share) {
  constexpr int BM = S::BM, BN = S::BN, kWaves = S::kWaves, kLoadsX = S::kLoadsX;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  lds_u8* const sm = (lds_u8*)(smem);

  int t_id = static_cast<int>(blockIdx.x & 7) * per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (t_id >= tiles_m * tiles_n * splits) return;
  const int split = kSplit ? t_id % splits : 0;
  if (kSplit) t_id /= splits;
  const int group_tiles = kGroupM * tiles_n;
  const int tgroup = t_id / group_tiles;
  const int first_m = tgroup * kGroupM;
  const int gm = min(kGroupM, tiles_m - first_m);
  const int in_group = t_id - tgroup * group_tiles;
  const int m0 = (first_m + in_group % gm) * BM;
  const int n0 = (in_group / gm) * BN;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int fi = lane & 31, fh = lane >> 5;

  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(xq + static_cast<size_t>(m0) * K, min(BM, M - m0) * K);
  const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(wq + static_cast<size_t>(n0) * K, min(BN, N - n0) * K);

  const int blocks = (K + kBK - 1) / kBK;
  const int first = kSplit ? split * share : 0, nst = kSplit ? min(share, blocks - first) : blocks;

  // A stage's scales come with its tiles, by the same kind of load: wavefronts
  // below BM / 64 bring those of 64 tokens each, the others those of the
  // channel blocks (lane r: block r of the tile), zeros past M and N. Loads
  // into registers would be waited for by count, and so for every fill before
  // them, however many stages ahead those are (48 tokens at K = 12288, N = 4096
  // were 13% slower so, 300 at 4096 x 4096 21%). (The addresses are uniform;
  // said, so that the loads need no loop over lanes.)
  const bool of_tokens = wave < BM / 64;
  const uint64_t scales_from = reinterpret_cast<uint64_t>(of_tokens ? s_x + static_cast<size_t>(first) * M + m0 + 64 * wave
                                                                    : s_w + static_cast<size_t>(n0 / 128) * blocks + first);
  const uint8_t* const scales = reinterpret_cast<const uint8_t*>(
      (static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(scales_from >> 32))) << 32) |
      static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(scales_from))));
  const uint32_t scale_step = __builtin_amdgcn_readfirstlane(of_tokens ? 4u * static_cast<uint32_t>(M) : 4u);
  const int scale_bytes = __builtin_amdgcn_readfirstlane(
      of_tokens ? 4 * min(max(M - m0 - 64 * wave, 0), 64) : 4 * (((min(BN, N - n0) + 127) / 128 - 1) * blocks + 1));
  const uint32_t scale_off = 4u * static_cast<uint32_t>(lane) * static_cast<uint32_t>(of_tokens ? 1 : blocks);
  const int scale_at = S::kTiles + (of_tokens ? 256 * wave : 4 * BM);

  // Fill l covers rows 8 (wave + kWaves l) .. + 7 of its operand's tile; lane L
  // writes physical chunk L % 8 of row L / 8, so it fetches the logical chunk
  // that the swizzle places there. The swizzle repeats every 16 rows, so the
  // fills of a lane differ by whole rows only.
  const int frow = 8 * wave + (lane >> 3);
  const int fk = 16 * ((lane & 7) ^ chunk_swizzle(frow));
  const uint32_t foff = static_cast<uint32_t>(frow * K + fk);
  auto fill = [&](int s) {
    const int k0 = (first + s) * kBK;
    const uint32_t base = fk < K - k0 ? foff : kOob;
    lds_u8* const dst = sm + (s % S::kSlots) * S::kStage + wave * 1024;
#pragma unroll
    for (int l = 0; l < S::kLoadsT; ++l) {
      const int u = l < kLoadsX ? l : l - kLoadsX;
      const uint32_t off = base + static_cast<uint32_t>(8 * kWaves * u * K + k0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          l < kLoadsX ? rx : rw, (lds_void*)(dst + (l < kLoadsX ? 0 : BM * kBK) + kWaves * u * 1024), 16, off, 0, 0, 0);
    }
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(scales + static_cast<uint64_t>(s) * scale_step, scale_bytes);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(sm + (s % S::kSlots) * S::kStage + scale_at), 4, scale_off, 0, 0,
                                             0);
  };

  // Fragment chunk c (0..3, two per k-step) of a row: logical chunk 2 c + fh.
  int coff[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) coff[c] = 16 * ((2 * c + fh) ^ chunk_swizzle(fi));
  const int xrow = (wm * 32 * S::TB + fi) * kBK;
  const int wrow = BM * kBK + (wn * 32 * S::TA + fi) * kBK;

  f32x16 acc[S::TA][S::TB];
#pragma unroll
  for (int a = 0; a < S::TA; ++a)
#pragma unroll
    for (int b = 0; b < S::TB; ++b) acc[a][b] = f32x16{};

  float sx[S::TB], sw = 0.f;
#pragma unroll
  for (int s = 0; s < S::kSlots - 1; ++s)
    if (s < nst) fill(s);
  if (S::kSlots - 1 <= nst) {
    wait_counts<S::kAhead, 0>();
  } else {
    wait_counts<0, 0>();
  }
  bare_barrier();

  auto fragment = [&](int slot, int at, int t) {
    const lds_u8* const src = sm + slot * S::kStage + at;
    const i32x4 lo = *(const lds_i32x4*)(src + coff[2 * t]);
    const i32x4 hi = *(const lds_i32x4*)(src + coff[2 * t + 1]);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto product = [&](const i32x8 (&w)[2], const i32x8 (&x)[2]) {
    f32x16 v = f32x16{};
    v = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[0], x[0], v, 0, 0, 0, 0, 0, 0);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[1], x[1], v, 0, 0, 0, 0, 0, 0);
  };
  auto add = [&](int a, int b, const f32x16& v) {
    const float sc = sx[b] * sw;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[a][b][i] = fmaf(v[i], sc, acc[a][b][i]);
  };
  // What every round s begins with: the fill of the stage kSlots - 1 ahead,
  // into the slot that every wavefront finished reading before the barrier
  // that ended round s - 1, and this stage's scales.
  auto begin = [&](int s) {
    if (s + S::kSlots - 1 < nst) fill(s + S::kSlots - 1);
    const lds_u8* const src = sm + (s % S::kSlots) * S::kStage + S::kTiles;
    sw = *(const lds_float*)(src + 4 * BM + 4 * (wn * 32 * S::TA / 128));
#pragma unroll
    for (int b = 0; b < S::TB; ++b) sx[b] = *(const lds_float*)(src + 4 * (wm * 32 * S::TB + 32 * b + fi));
  };
  // And ends with: this wavefront's share of the next stage needed is there.
  auto end = [&](int s) {
    if (s + S::kSlots - 1 < nst) {
      wait_counts<S::kAhead, 0>();
    } else {
      wait_counts<0, 0>();
    }
    bare_barrier();
  };

  if constexpr (S::TA * S::TB <= 4) {
    for (int s = 0; s < nst; ++s) {
      begin(s);
      const int slot = s % S::kSlots;
      i32x8 fw[S::TA][2], fx[S::TB][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int a = 0; a < S::TA; ++a) fw[a][t] = fragment(slot, wrow + a * 32 * kBK, t);
#pragma unroll
        for (int b = 0; b < S::TB; ++b) fx[b][t] = fragment(slot, xrow + b * 32 * kBK, t);
      }
#pragma unroll
      for (int a = 0; a < S::TA; ++a)
#pragma unroll
        for (int b = 0; b < S::TB; ++b) add(a, b, product(fw[a], fx[b]));
      end(s);
    }
  } else {
    // Large wavefront tiles: the next token tile's fragments are read under
    // this one's MFMAs, a tile's multiply-adds follow the next tile's MFMAs.
    // The fences and the empty statement hold that order: left alone the
    // compiler moves every multiply-add behind the round, where the products
    // no longer fit the registers.
    for (int s = 0; s < nst; ++s) {
      begin(s);
      const int slot = s % S::kSlots;
      i32x8 fw[S::TA][2], fx[2][2];
      f32x16 p[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int a = 0; a < S::TA; ++a) fw[a][t] = fragment(slot, wrow + a * 32 * kBK, t);
        fx[0][t] = fragment(slot, xrow, t);
      }
#pragma unroll
      for (int at = 0; at < S::TA * S::TB; ++at) {
        const int b = at / S::TA, a = at % S::TA;
        if (a == 0 && b + 1 < S::TB) {
#pragma unroll
          for (int t = 0; t < 2; ++t) fx[(b + 1) & 1][t] = fragment(slot, xrow + (b + 1) * 32 * kBK, t);
        }
        p[at & 1] = product(fw[a], fx[b & 1]);
        if (at > 0) {
          const int b1 = (at - 1) / S::TA, a1 = (at - 1) % S::TA;
          add(a1, b1, p[(at - 1) & 1]);
          asm volatile("" : "+v"(acc[a1][b1]));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      add(S::TA - 1, S::TB - 1, p[(S::TA * S::TB - 1) & 1]);
      end(s);
    }
  }

  // Lane (j, h) register r of a tile holds channel 8 (r / 4) + 4 h + r % 4 of
  // token j.
  if constexpr (kSplit) {
#pragma unroll
    for (int b = 0; b < S::TB; ++b) {
      const int m = m0 + wm * 32 * S::TB + 32 * b + fi;
      if (m >= M) continue;
      float* const row = part + (static_cast<size_t>(split) * M + m) * N;
#pragma unroll
      for (int a = 0; a < S::TA; ++a)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn * 32 * S::TA + 32 * a + 8 * q + 4 * fh;
          if ((N & 3) == 0) {
            if (n < N)
              *reinterpret_cast<f32x4*>(row + n) =
                  f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < N) row[n + i] = acc[a][b][4 * q + i];
          }
        }
    }
    return;
  }
  // Staged in LDS as rows of 16-bit outputs, written out whole.
#pragma unroll
  for (int a = 0; a < S::TA; ++a)
#pragma unroll
    for (int b = 0; b < S::TB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = wm * 32 * S::TB + 32 * b + fi, col = wn * 32 * S::TA + 32 * a + 8 * q + 4 * fh;
        uint32_t hv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) hv[i] = half_bits<kBf16>(acc[a][b][4 * q + i]);
        *(lds_u32x2*)(sm + row * S::kPitch + col * 2) = u32x2{hv[0] | (hv[1] << 16), hv[2] | (hv[3] << 16)};
      }
  wait_counts<0, 0>();
  bare_barrier();
  constexpr int kPieces = BN * 2 / 16;  // 16-byte pieces per row
  const int c = threadIdx.x % kPieces;
  const int n = n0 + 8 * c;
  const bool whole = (N & 7) == 0;  // rows start 16-byte aligned; a piece is all in or all out
  for (int rr = threadIdx.x / kPieces; rr < BM; rr += S::kThreads / kPieces) {
    const int m = m0 + rr;
    if (m >= M || n >= N) continue;
    const u32x4 v = *(const lds_u32x4*)(sm + rr * S::kPitch + c * 16);
    uint16_t* const o = y + static_cast<size_t>(m) * N + n;
    if (whole) {
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(o));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (n + i >= N) break;
        o[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2)));
      }
    }
  }
}

// Adds the splits of every output in split order.
template <bool kBf16>
__global__ __launch_bounds__(256) void fp8_join_kernel(const float* __restrict__ part, uint16_t* __restrict__ y,
                                                       int64_t outputs, int splits) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at + 4 <= outputs && (outputs & 3) == 0) {
    f32x4 v = *reinterpret_cast<const f32x4*>(part + at);
    for (int z0 = 1; z0 < splits; z0 += 4) {  // four loads at a time
      f32x4 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        p[u] = z0 + u < splits ? *reinterpret_cast<const f32x4*>(part + (z0 + u) * outputs + at) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = z0 + u < splits ? v[i] + p[u][i] : v[i];
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = half_bits<kBf16>(v[i]);
    *reinterpret_cast<u32x2*>(y + at) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    return;
  }
  for (int64_t o = at; o < at + 4 && o < outputs; ++o) {
    float v = part[o];
    for (int z = 1; z < splits; ++z) v += part[z * outputs + o];
    y[o] = half_bits<kBf16>(v);
  }
}

template <typename S>
hipError_t launch_shape(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y, int M,
                        int N, int K, int splits, float* part, bool bf16, hipStream_t stream) {
  const int tiles_m = (M + S::BM - 1) / S::BM, tiles_n = (N + S::BN - 1) / S::BN;
  const int blocks = (K + kBK - 1) / kBK, share = (blocks + splits - 1) / splits;
  const int64_t units = static_cast<int64_t>(tiles_m) * tiles_n * splits;
  if (units > (1 << 22) || share * (splits - 1) >= blocks) return hipErrorInvalidValue;
  const int per_xcd = static_cast<int>((units + 7) / 8);
  const dim3 grid(static_cast<uint32_t>(8 * per_xcd)), block(S::kThreads);
  if (splits == 1) {
    if (bf16)
      return launch_kernel(fp8_block_mm_kernel<S, false, true>, grid, block, 0, stream, xq, s_x, wq, s_w, y, part, M, N,
                           K, tiles_m, tiles_n, per_xcd, 1, blocks);
    return launch_kernel(fp8_block_mm_kernel<S, false, false>, grid, block, 0, stream, xq, s_x, wq, s_w, y, part, M, N,
                         K, tiles_m, tiles_n, per_xcd, 1, blocks);
  }
  const hipError_t e = launch_kernel(fp8_block_mm_kernel<S, true, false>, grid, block, 0, stream, xq, s_x, wq, s_w, y,
                                     part, M, N, K, tiles_m, tiles_n, per_xcd, splits, share);
  if (e != hipSuccess) return e;
  const int64_t outputs = static_cast<int64_t>(M) * N;
  const dim3 jgrid(static_cast<uint32_t>((outputs + 1023) / 1024));
  if (bf16) return launch_kernel(fp8_join_kernel<true>, jgrid, dim3(256), 0, stream, part, y, outputs, splits);
  return launch_kernel(fp8_join_kernel<false>, jgrid, dim3(256), 0, stream, part, y, outputs, splits);
}

typedef Shape<256, 256, 2, 4, 2> Big;
typedef Shape<128, 128, 2, 2, 2> Mid;   // two workgroups per CU, here and below
typedef Shape<64, 128, 2, 2, 3> Low;
typedef Shape<64, 64, 2, 2, 4> Small;

}  // namespace

// Which tile, and how many ranges of K. A tile's stages cost the more the
// larger it is, a launch takes as many of them as its fullest CU holds, and
// splitting K adds a second kernel and the sums' way through memory. The
// figures (microseconds) are fitted to timed launches of every form over 17 to
// 4096 tokens: per stage with one workgroup on a CU, with two of them, and what
// a split adds. For example 48 tokens at K = 12288, N = 4096: 64 x 64 tiles in 4
// ranges 14.8 us, in 8 15.9, 64 x 128 in 8 15.4; 300 tokens at 4096 x 4096: 64 x
// 64 15.8, in 2 ranges 21.1, 64 x 128 19.8; 517 at 4096 x 6144: 64 x 128 26.0
// (128 x 64, which is not among the forms, 26.2, and behind the quantizer 29.7
// like it), 64 x 64 33.0, 128 x 128 31.2; 2048 at 4096 x 4096: 128 x 128 40.7,
// 64 x 128 53.2, 256 x 256 60.2; 4096 at 4096 x 24576: 256 x 256 407, 128 x 128
// 473, 64 x 128 583.
Fp8Plan plan_fp8_block_mm(int64_t M, int64_t N, int64_t K) {
  Fp8Plan p = {Fp8Form::kGemv, 1, 0};
  if (fp8_use_gemv(M, K)) return p;
  struct Cost {
    Fp8Form form;
    int bm, bn;
    double one, two;
  };
  constexpr Cost kCosts[] = {{Fp8Form::kBig, 256, 256, 1.75, 3.5},
                             {Fp8Form::kMid, 128, 128, 0.82, 0.90},
                             {Fp8Form::kLow, 64, 128, 0.54, 0.64},
                             {Fp8Form::kSmall, 64, 64, 0.33, 0.45}};
  const int64_t blocks = (K + kBK - 1) / kBK;
  double best = 1e300;
  for (const Cost& c : kCosts) {
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      const int64_t share = (blocks + splits - 1) / splits;
      if (splits > 1 && (share * (splits - 1) >= blocks || tiles * splits > 1024)) break;
      const int64_t on = (tiles * splits + 255) / 256;  // workgroups of the fullest CU
      double t = static_cast<double>(share) * (static_cast<double>(on / 2) * c.two + static_cast<double>(on % 2) * c.one);
      if (splits > 1) t += 2.0 + static_cast<double>(splits) * (0.5 + static_cast<double>(M * N) * 1.6e-6);
      if (t < best) {
        best = t;
        p.form = c.form;
        p.splits = splits;
      }
    }
  }
  if (p.splits > 1) p.workspace_bytes = static_cast<size_t>(p.splits) * static_cast<size_t>(M * N) * sizeof(float);
  return p;
}

hipError_t launch_fp8_block_mm(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                               int64_t M, int64_t N, int64_t K, const Fp8Plan& plan, void* workspace, bool bf16,
                               hipStream_t stream) {
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  float* const part = static_cast<float*>(workspace);
  switch (plan.form) {
    case Fp8Form::kGemv: return launch_fp8_block_gemv(nullptr, xq, s_x, wq, s_w, y, M, N, K, bf16, stream);
    case Fp8Form::kBig: return launch_shape<Big>(xq, s_x, wq, s_w, y, m, n, k, plan.splits, part, bf16, stream);
    case Fp8Form::kMid: return launch_shape<Mid>(xq, s_x, wq, s_w, y, m, n, k, plan.splits, part, bf16, stream);
    case Fp8Form::kLow: return launch_shape<Low>(xq, s_x, wq, s_w, y, m, n, k, plan.splits, part, bf16, stream);
    case Fp8Form::kSmall: return launch_shape<Small>(xq, s_x, wq, s_w, y, m, n, k, plan.splits, part, bf16, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace mq
