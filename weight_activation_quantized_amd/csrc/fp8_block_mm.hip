// e4m3 matrix product with one scale per block of 128, for gfx950 (more than
// 64 tokens; fp8_block_gemv.hip takes the rest).
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
//   to parity with the MFMAs), and each SIMD has two wavefronts so that one's
//   multiply-adds run under the other's MFMAs.
// - Weight rows are the MFMA's A operand and token rows its B operand: a lane
//   of the 32x32 result holds one token, so the scale sx * sw is one value
//   per lane and tile (sw is uniform: a tile of 32 channels lies within one
//   block of 128).
// - Tiles move HBM -> LDS by buffer_load ... lds, one stage of 128 bytes of K
//   ahead of the compute. LDS rows are 128 bytes, their 16-byte chunks
//   XOR-swizzled by the row, so a fragment read of 32 rows meets no bank
//   conflict. Loads past the buffer's end return zero (ragged M, N, K).
// - A lane's 32 bytes of a k-step are the chunks 4 t + h and 4 t + 2 + h of
//   its row; which k a lane holds does not matter as long as both operands
//   agree.
// - Workgroups go round-robin over the 8 XCDs; each XCD gets a contiguous run
//   of tiles in groups of kGroupM token tiles, so that what a run shares stays
//   in its L2.
#include "device_common.h"
#include "launch.h"

namespace mq {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int kBK = 128;  // bytes of K per stage: one scale block
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kGroupM = 4;                // token tiles per group in the tile order
constexpr uint32_t kOob = 0x80000000u;    // a buffer offset past every tile: the load returns 0
constexpr int kBufferFlags = 0x00020000;  // gfx9 buffer descriptor word 3 (raw 32-bit data)

__device__ __forceinline__ int chunk_swizzle(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, kBufferFlags);
}

// A workgroup computes BM tokens x BN channels; its eight wavefronts stand WM
// x WN over it, each with a tile of 32 TB tokens x 32 TA channels.
template <int BM, int BN, int WM>
struct Shape {
  static constexpr int WN = kWaves / WM;
  static constexpr int TB = BM / WM / 32, TA = BN / WN / 32;
  static constexpr int kStage = (BM + BN) * kBK;
  static constexpr int kSlots = 3 * kStage <= 150 * 1024 ? 3 : 2;
  static constexpr int kPitch = BN * 2 + 16;  // staged output rows
  static constexpr int kLds = kSlots * kStage > BM * kPitch ? kSlots * kStage : BM * kPitch;
  static constexpr int kLoads = (BM + BN) / 8 / kWaves;  // fills per wavefront and stage (8 rows of 128 bytes each)
  static_assert(kLds <= 160 * 1024, "LDS capacity");
  static_assert(TA >= 1 && TB >= 1 && (BM + BN) % (8 * kWaves) == 0 && BN % 128 == 0, "tile shape");
  static_assert(BM % (8 * kWaves) == 0, "a wavefront's fills do not straddle the operands");
};

template <int BM, int BN, int WM, bool kBf16>
__global__ __launch_bounds__(kThreads) void fp8_block_mm_kernel(
    const uint8_t* __restrict__ xq, const float* __restrict__ s_x, const uint8_t* __restrict__ wq,
    const float* __restrict__ s_w, uint16_t* __restrict__ y, int M, int N, int K, int tiles_m, int tiles_n,
    int per_xcd) {
  typedef Shape<BM, BN, WM> S;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  lds_u8* const sm = (lds_u8*)(smem);

  const int t_id = static_cast<int>(blockIdx.x & 7) * per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (t_id >= tiles_m * tiles_n) return;
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

  // Fill l covers tile rows 8 (wave + 8 l) .. + 7 (token rows first, then
  // channel rows); lane L writes physical chunk L % 8 of row L / 8, so it
  // fetches the logical chunk that the swizzle places there.
  constexpr int kLoadsX = BM / 8 / kWaves;
  uint32_t loff[S::kLoads];
  int lk[S::kLoads];
#pragma unroll
  for (int l = 0; l < S::kLoads; ++l) {
    const int row = 8 * (wave + kWaves * (l < kLoadsX ? l : l - kLoadsX)) + (lane >> 3);
    lk[l] = 16 * ((lane & 7) ^ chunk_swizzle(row));
    loff[l] = static_cast<uint32_t>(row * K + lk[l]);
  }
  auto fill = [&](int s) {
    const int k0 = s * kBK;
    const int krem = K - k0;
    lds_u8* const dst = sm + (s % S::kSlots) * S::kStage;
#pragma unroll
    for (int l = 0; l < S::kLoads; ++l) {
      const uint32_t off = lk[l] < krem ? loff[l] + k0 : kOob;
      if (l < kLoadsX) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(dst + (wave + kWaves * l) * 1024), 16, off, 0, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rw, (lds_void*)(dst + BM * kBK + (wave + kWaves * (l - kLoadsX)) * 1024), 16, off, 0, 0, 0);
      }
    }
  };

  // Fragment chunk c (0..3, two per k-step) of a row: logical chunk 2 c + fh.
  int coff[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) coff[c] = 16 * ((2 * c + fh) ^ chunk_swizzle(fi));
  const int xrow = (wm * 32 * S::TB + fi) * kBK;
  const int wrow = BM * kBK + (wn * 32 * S::TA + fi) * kBK;

  // Scales: this lane's token of each 32-token tile (tokens past M take the
  // last one's; their results are not stored), this wavefront's channel block.
  const int nst = (K + kBK - 1) / kBK;
  int tok[S::TB];
#pragma unroll
  for (int b = 0; b < S::TB; ++b) tok[b] = min(m0 + wm * 32 * S::TB + 32 * b + fi, M - 1);
  int nblk[S::TA];
#pragma unroll
  for (int a = 0; a < S::TA; ++a) nblk[a] = min(n0 + wn * 32 * S::TA + 32 * a, N - 1) / 128;

  f32x16 acc[S::TA][S::TB];
#pragma unroll
  for (int a = 0; a < S::TA; ++a)
#pragma unroll
    for (int b = 0; b < S::TB; ++b) acc[a][b] = f32x16{};

  float sx[S::TB], sw[S::TA], sxn[S::TB], swn[S::TA];
#pragma unroll
  for (int b = 0; b < S::TB; ++b) sx[b] = s_x[tok[b]];
#pragma unroll
  for (int a = 0; a < S::TA; ++a) sw[a] = s_w[static_cast<size_t>(nblk[a]) * nst];

  fill(0);
  if (S::kSlots > 2 && nst > 1) fill(1);
  if (S::kSlots > 2 && nst > 1) {
    wait_counts<S::kLoads, 0>();
  } else {
    wait_counts<0, 0>();
  }
  bare_barrier();

  // Round s: the scales of stage s + 1 and the fill of the stage kSlots - 1
  // ahead go out (into the slot that every wavefront finished reading before
  // the barrier that ended round s - 1), stage s is computed, and the
  // wavefront waits for its own share of stage s + 1 before the barrier.
  for (int s = 0; s < nst; ++s) {
    const int s1 = min(s + 1, nst - 1);
#pragma unroll
    for (int b = 0; b < S::TB; ++b) sxn[b] = s_x[static_cast<size_t>(s1) * M + tok[b]];
#pragma unroll
    for (int a = 0; a < S::TA; ++a) swn[a] = s_w[static_cast<size_t>(nblk[a]) * nst + s1];
    const bool more = s + S::kSlots - 1 < nst;
    if (more) fill(s + S::kSlots - 1);

    const lds_u8* const src = sm + (s % S::kSlots) * S::kStage;
    i32x8 fw[S::TA][2];
#pragma unroll
    for (int a = 0; a < S::TA; ++a)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const i32x4 lo = *(const lds_i32x4*)(src + wrow + a * 32 * kBK + coff[2 * t]);
        const i32x4 hi = *(const lds_i32x4*)(src + wrow + a * 32 * kBK + coff[2 * t + 1]);
        fw[a][t] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
#pragma unroll
    for (int b = 0; b < S::TB; ++b) {
      i32x8 fx[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const i32x4 lo = *(const lds_i32x4*)(src + xrow + b * 32 * kBK + coff[2 * t]);
        const i32x4 hi = *(const lds_i32x4*)(src + xrow + b * 32 * kBK + coff[2 * t + 1]);
        fx[t] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
#pragma unroll
      for (int a = 0; a < S::TA; ++a) {
        f32x16 p = f32x16{};
        p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[a][0], fx[0], p, 0, 0, 0, 0, 0, 0);
        p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[a][1], fx[1], p, 0, 0, 0, 0, 0, 0);
        const float sc = sx[b] * sw[a];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = fmaf(p[i], sc, acc[a][b][i]);
      }
    }
#pragma unroll
    for (int b = 0; b < S::TB; ++b) sx[b] = sxn[b];
#pragma unroll
    for (int a = 0; a < S::TA; ++a) sw[a] = swn[a];
    if (S::kSlots > 2 && more) {
      wait_counts<S::kLoads, 0>();
    } else {
      wait_counts<0, 0>();
    }
    bare_barrier();
  }

  // Lane (j, h) register r of a tile holds channel 8 (r / 4) + 4 h + r % 4 of
  // token j: staged in LDS as rows of 16-bit outputs, written out whole.
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
  for (int rr = threadIdx.x / kPieces; rr < BM; rr += kThreads / kPieces) {
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

template <int BM, int BN, int WM>
hipError_t launch_shape(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y, int M,
                        int N, int K, bool bf16, hipStream_t stream) {
  const int tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
  const int64_t tiles = static_cast<int64_t>(tiles_m) * tiles_n;
  if (tiles > (1 << 22)) return hipErrorInvalidValue;
  const int per_xcd = static_cast<int>((tiles + 7) / 8);
  const dim3 grid(static_cast<uint32_t>(8 * per_xcd)), block(kThreads);
  if (bf16)
    return launch_kernel(fp8_block_mm_kernel<BM, BN, WM, true>, grid, block, 0, stream, xq, s_x, wq, s_w, y, M, N, K,
                         tiles_m, tiles_n, per_xcd);
  return launch_kernel(fp8_block_mm_kernel<BM, BN, WM, false>, grid, block, 0, stream, xq, s_x, wq, s_w, y, M, N, K,
                       tiles_m, tiles_n, per_xcd);
}

}  // namespace

hipError_t launch_fp8_block_mm(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                               int64_t M, int64_t N, int64_t K, bool bf16, hipStream_t stream) {
  if (M <= kFp8GemvMaxM) return launch_fp8_block_gemv(xq, s_x, wq, s_w, y, M, N, K, bf16, stream);
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  const int64_t big = ((M + 255) / 256) * ((N + 255) / 256);
  if (big >= 200) return launch_shape<256, 256, 2>(xq, s_x, wq, s_w, y, m, n, k, bf16, stream);
  const int64_t mid = ((M + 255) / 256) * ((N + 127) / 128);
  if (mid >= 200) return launch_shape<256, 128, 4>(xq, s_x, wq, s_w, y, m, n, k, bf16, stream);
  return launch_shape<64, 128, 2>(xq, s_x, wq, s_w, y, m, n, k, bf16, stream);
}

}  // namespace mq
