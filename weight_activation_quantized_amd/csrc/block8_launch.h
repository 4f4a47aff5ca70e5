// Launchers of the 8-bit attention block: RMS norm with 8-bit output, e4m3
// quantizer and product, paged e4m3 KV cache. Apart from launch.h, so that a
// change here leaves the other kernels' sources as they are.
#pragma once

#include "launch.h"

namespace mq {

// RMS norm of x (+ residual, the sum stored in h) [M, K] with 8-bit output:
// int8 codes and one scale per row, or, when fp8, e4m3 codes and one scale per
// 128 values, scales [ceil(K / 128), M]. residual and h are NULL together; h
// may be residual itself. Rows stay in registers: K <= kRmsnormMaxK.
constexpr int64_t kRmsnormMaxK = 65536;
hipError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps,
                                uint16_t* h, uint8_t* codes, float* scales, int64_t M, int64_t K, bool fp8, bool bf16,
                                hipStream_t stream);

// e4m3 codes [M, K] of x and one scale per 128 values, scales [ceil(K / 128), M].
hipError_t launch_quant_fp8_blocks(const uint16_t* x, uint8_t* codes, float* scales, int64_t M, int64_t K, bool bf16,
                                   hipStream_t stream);

// y[M, N] = xq[M, K] . wq[N, K]^T, both e4m3 with scales per block of 128
// (s_x [ceil(K / 128), M], s_w [ceil(N / 128), ceil(K / 128)]); the form for
// few tokens where fp8_use_gemv says.
enum class Fp8Form { kGemv, kSmall, kLow, kMid, kBig };
struct Fp8Plan {
  Fp8Form form;
  int splits;              // ranges of K, each a workgroup's; their sums meet in the workspace
  size_t workspace_bytes;  // 0 without splits
};
Fp8Plan plan_fp8_block_mm(int64_t M, int64_t N, int64_t K);
hipError_t launch_fp8_block_mm(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                               int64_t M, int64_t N, int64_t K, const Fp8Plan& plan, void* workspace, bool bf16,
                               hipStream_t stream);

// The form for few tokens whose codes fit LDS; with x (and without xq, s_x) it
// quantizes the rows itself, to the same bits, where fp8_use_fused says.
bool fp8_use_gemv(int64_t M, int64_t K);
bool fp8_use_fused(int64_t M, int64_t K);
hipError_t launch_fp8_block_gemv(const uint16_t* x, const uint8_t* xq, const float* s_x, const uint8_t* wq,
                                 const float* s_w, uint16_t* y, int64_t M, int64_t N, int64_t K, bool bf16,
                                 hipStream_t stream);

// The paged e4m3 KV cache: K pages [page, head_dim] and V pages
// [head_dim, page] for every (page, kv head), one binary32 scale each; the
// sequences' page tables and lengths, which only the GPU reads.
struct Kv8Cache {
  uint8_t* k;
  uint8_t* v;
  float* k_scales;  // [num_pages, kv_heads]
  float* v_scales;
  const int32_t* table;  // [batch, table_width]
  const int32_t* cu;     // [batch + 1]: first row of each sequence's new tokens
  const int32_t* lens;   // [batch]: tokens in the cache, the new ones included
  int batch, kv_heads, head_dim, page, num_pages, table_width;
  int page_shift;  // page = 1 << page_shift (16, 32, 64 or 128 tokens)
  int tokens;     // rows of q / k / v
  int max_q_len;  // at least every sequence's number of new tokens
};

// Writes rows k, v [tokens, kv_heads, head_dim] (stride elements between
// tokens) into the pages of their sequences.
int64_t kv8_append_blocks(const Kv8Cache& c);  // workgroups of the launch
hipError_t launch_kv8_append(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                             int64_t v_stride, bool bf16, hipStream_t stream);

// out [tokens, q_heads, head_dim] = causal attention of q over the cache. With
// plan.splits > 1 every split of the keys leaves its part in the workspace and
// a second kernel joins them.
struct Kv8Plan {
  bool decode;  // the rows of one kv head fit a few tiles of 16: the streaming form
  int waves;    // wavefronts of a workgroup
  int splits;
  int64_t prompt_blocks;  // workgroups of the other form (under 2^29 within the entry's limits)
  size_t workspace_bytes;
};
Kv8Plan plan_kv8_attention(const Kv8Cache& c, int q_heads);
hipError_t launch_kv8_attention(const Kv8Cache& c, const uint16_t* q, int64_t q_stride, uint16_t* out, int q_heads,
                                float softmax_scale, const Kv8Plan& plan, void* workspace, bool bf16,
                                hipStream_t stream);

}  // namespace mq
