// e4m3 matrix product with one scale per block of 128 for up to 64 tokens, on
// gfx950. Same definition as fp8_block_mm.hip:
//
//   y[m,n] = rne16( sum_b (sx[b,m] * sw[n/128,b]) * sum_{k in block b} xq[m,k] * wq[n,k] )
//
// (the fp8 matrix unit's alignment of 8 products as described there).
//
// With few tokens the product is bound by the weight stream (N*K bytes), so
// every weight byte is read once, straight into registers, with as many bytes
// in flight as the registers hold:
// - A workgroup owns 16 output channels; its wavefronts split K into
//   contiguous ranges of whole blocks and add their binary32 sums in LDS in
//   wavefront order (deterministic).
// - v_mfma_f32_16x16x128_f8f6f4 covers exactly one scale block: weight rows
//   are its A operand, 16 tokens its B operand. Lane (i = lane % 16,
//   h = lane / 16) takes the 16-byte chunks h and 4 + h of row i's 128 bytes
//   (both operands alike, so which k a lane holds does not matter): the four
//   lanes of a row read 64 contiguous bytes. The block's result starts from
//   zero and joins the running sum with four multiply-adds per lane.
// - Two register sets of blocks alternate: one set's loads are in flight while
//   the other's MFMAs run. Buffer loads past a descriptor's size return zero
//   (rows past N, tokens past M, the end of a ragged last block).
#include "device_common.h"
#include "launch.h"

namespace mq {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOob = 0x80000000u;    // a buffer offset past every operand: the load returns 0
constexpr int kBufferFlags = 0x00020000;  // gfx9 buffer descriptor word 3 (raw 32-bit data)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  const int64_t n = bytes < 0 ? 0 : (bytes > 0x7fffffff ? 0x7fffffff : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(n), kBufferFlags);
}

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// One register set: kU blocks of one 16-channel weight tile and kT 16-token
// tiles, with the token scales of each.
template <int kU, int kT>
struct Set {
  i32x4 w[kU][2], x[kU][kT][2];
  float sx[kU][kT], sw[kU];
};

template <int kU, int kT>
__device__ __forceinline__ void issue(Set<kU, kT>& f, __amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rx,
                                      __amdgpu_buffer_rsrc_t rsx, const float* __restrict__ s_w, int i, int h, int M,
                                      int K, int b0, int b_end) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int b = b0 + u;
    const bool in = b < b_end;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = 128 * b + 64 * c + 16 * h;
      const bool ok = in && k < K;
      f.w[u][c] = load16(rw, ok ? static_cast<uint32_t>(i * K + k) : kOob);
#pragma unroll
      for (int t = 0; t < kT; ++t) f.x[u][t][c] = load16(rx, ok ? static_cast<uint32_t>((16 * t + i) * K + k) : kOob);
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const bool ok = in && 16 * t + i < M;
      f.sx[u][t] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(rsx, ok ? static_cast<uint32_t>(b * M + 16 * t + i) * 4u : kOob,
                                                      0, 0));
    }
    f.sw[u] = s_w[in ? b : b_end - 1];
  }
}

template <int kU, int kT>
__device__ __forceinline__ void use(const Set<kU, kT>& f, f32x4 (&acc)[kT]) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const i32x8 w = __builtin_shufflevector(f.w[u][0], f.w[u][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const i32x8 x = __builtin_shufflevector(f.x[u][t][0], f.x[u][t][1], 0, 1, 2, 3, 4, 5, 6, 7);
      f32x4 p = {0.f, 0.f, 0.f, 0.f};
      p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, p, 0, 0, 0, 0, 0, 0);
      const float sc = f.sx[u][t] * f.sw[u];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(p[e], sc, acc[t][e]);
    }
  }
}

template <int kW, int kU, int kT, bool kBf16>
__global__ __launch_bounds__(64 * kW) void fp8_block_gemv_kernel(const uint8_t* __restrict__ xq,
                                                                 const float* __restrict__ s_x,
                                                                 const uint8_t* __restrict__ wq,
                                                                 const float* __restrict__ s_w,
                                                                 uint16_t* __restrict__ y, int M, int N, int K) {
  __shared__ float part[kW][16 * kT][17];
  const int n0 = static_cast<int>(blockIdx.x) * 16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, h = lane >> 4;
  const int blocks = (K + 127) / 128;
  const int share = (blocks + kW - 1) / kW;
  const int b_begin = min(blocks, wave * share), b_end = min(blocks, b_begin + share);

  const __amdgpu_buffer_rsrc_t rw = rsrc(wq + static_cast<size_t>(n0) * K, static_cast<int64_t>(min(16, N - n0)) * K);
  const __amdgpu_buffer_rsrc_t rx = rsrc(xq, static_cast<int64_t>(M) * K);
  const __amdgpu_buffer_rsrc_t rsx = rsrc(s_x, static_cast<int64_t>(blocks) * M * 4);
  const float* const sw = s_w + static_cast<size_t>(n0 / 128) * blocks;

  f32x4 acc[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (b_begin < b_end) {
    Set<kU, kT> fa, fb;
    issue(fa, rw, rx, rsx, sw, i, h, M, K, b_begin, b_end);
    for (int b = b_begin; b < b_end; b += 2 * kU) {
      issue(fb, rw, rx, rsx, sw, i, h, M, K, b + kU, b_end);
      __builtin_amdgcn_sched_barrier(0);
      use(fa, acc);
      __builtin_amdgcn_sched_barrier(0);
      issue(fa, rw, rx, rsx, sw, i, h, M, K, b + 2 * kU, b_end);
      __builtin_amdgcn_sched_barrier(0);
      use(fb, acc);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Lane (j, h) register e of a tile holds channel 4 h + e of token j.
#pragma unroll
  for (int t = 0; t < kT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][16 * t + i][4 * h + e] = acc[t][e];
  __syncthreads();
  for (int o = threadIdx.x; o < 256 * kT; o += 64 * kW) {
    const int m = o >> 4, n = o & 15;
    float v = part[0][m][n];
#pragma unroll
    for (int w = 1; w < kW; ++w) v += part[w][m][n];
    if (m < M && n0 + n < N) y[static_cast<size_t>(m) * N + n0 + n] = half_bits<kBf16>(v);
  }
}

template <int kW, int kU, int kT>
hipError_t launch_tiles(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y, int M,
                        int N, int K, bool bf16, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((N + 15) / 16)), block(64 * kW);
  if (bf16)
    return launch_kernel(fp8_block_gemv_kernel<kW, kU, kT, true>, grid, block, 0, stream, xq, s_x, wq, s_w, y, M, N, K);
  return launch_kernel(fp8_block_gemv_kernel<kW, kU, kT, false>, grid, block, 0, stream, xq, s_x, wq, s_w, y, M, N, K);
}

}  // namespace

hipError_t launch_fp8_block_gemv(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                                 int64_t M, int64_t N, int64_t K, bool bf16, hipStream_t stream) {
  if (M > kFp8GemvMaxM) return hipErrorInvalidValue;
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  if (M <= 16) return launch_tiles<8, 2, 1>(xq, s_x, wq, s_w, y, m, n, k, bf16, stream);
  if (M <= 32) return launch_tiles<8, 2, 2>(xq, s_x, wq, s_w, y, m, n, k, bf16, stream);
  return launch_tiles<8, 1, 4>(xq, s_x, wq, s_w, y, m, n, k, bf16, stream);
}

}  // namespace mq
