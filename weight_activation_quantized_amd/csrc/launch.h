// Internal launcher declarations shared by the C-ABI layer (mq_api.cpp) and
// the kernel translation units. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace mq {

// Per-token int8 quantization of x[M,K] (fp16, or bf16 when bf16) into
// xq[M,K] and s_tok[M].
hipError_t launch_quant_per_token_int8(const uint16_t* x, int8_t* xq, float* s_tok, int64_t M, int64_t K, bool bf16,
                                       hipStream_t stream);

// int8 GEMM acc = xq[M,K] . wq[N,K]^T. Exactly one of y (scaled output,
// fp16 or, when bf16, bf16; needs s_tok and s_ch) and acc (raw int32 output)
// is non-null.
hipError_t launch_w8a8_gemm(const int8_t* xq, const float* s_tok, const int8_t* wq,
                            const float* s_ch, uint16_t* y, int32_t* acc,
                            int64_t M, int64_t N, int64_t K, bool bf16, hipStream_t stream);

// Decode-shaped form of the same product (M <= kW8A8GemvMaxM), bound by the
// weight stream; launch_w8a8_gemm dispatches to it where w8a8_use_gemv says.
constexpr int64_t kW8A8GemvMaxM = 64;
bool w8a8_use_gemv(int64_t M, int64_t N);
hipError_t launch_w8a8_gemv(const int8_t* xq, const float* s_tok, const int8_t* wq,
                            const float* s_ch, uint16_t* y, int32_t* acc,
                            int64_t M, int64_t N, int64_t K, bool bf16, hipStream_t stream);

// Quantizer folded into the decode kernel: y = scaled_mm(quant(x), wq, s_ch)
// in one launch, bit-identical to the two separate calls, where
// w8a8_use_fused(M, N, K): one token with K <= 12288, two with K <= 8192,
// three or four with K <= 4096 and N >= 6144 (the token rows held in a
// 256-thread workgroup's registers). Every workgroup forms the tokens'
// scales and codes itself, once for all its tiles, while its first weight
// requests are in flight, which beats the quantizer launch there.
bool w8a8_use_fused(int64_t M, int64_t N, int64_t K);
hipError_t launch_w8a8_gemv_fused(const uint16_t* x, const int8_t* wq, const float* s_ch, uint16_t* y,
                                  int64_t M, int64_t N, int64_t K, bool bf16, hipStream_t stream);

// Device address of the library-owned scratch array on the current device
// (looked up once per device), kNoallocScratchBytes long, 256-byte aligned.
constexpr size_t kNoallocScratchBytes = 33816576;  // MQ_NOALLOC_SCRATCH_BYTES
hipError_t noalloc_scratch(void** ptr);

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
// (s_x [ceil(K / 128), M], s_w [ceil(N / 128), ceil(K / 128)]); the decode
// form for M <= kFp8GemvMaxM.
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

// Online KV-cache quantization of rows x [rows, head_dim] fp16 to codes
// (uint8 [rows, head_dim] for 8 bits, packed [rows, head_dim/2] for 4) and
// params fp32 [rows, 2] = (scale, min); head_dim a power of two in [8, 512];
// x is fp16, or bf16 when bf16.
hipError_t launch_kv_quant(const uint16_t* x, uint8_t* codes, float* params, int64_t rows, int64_t head_dim,
                           int bits, bool bf16, hipStream_t stream);

// Checkpoint-layout adapter (one-time conversions, exact bit permutations).
// order[j] = the element (0..7 within the word's span) that field j of a
// source word holds; the result is in the library's order (field j = element j).
hipError_t launch_int4_reorder(const int32_t* src, int32_t* dst, int64_t words, const uint8_t (&order)[8],
                               hipStream_t stream);
// src [A, B/8] packed along B in `order` -> dst [B, A/8] packed along A.
hipError_t launch_int4_transpose(const int32_t* src, int32_t* dst, int64_t A, int64_t B, const uint8_t (&order)[8],
                                 hipStream_t stream);
constexpr int64_t kInt4TransposeMaxA = int64_t{65535} * 128;
// src [A, B] 16-bit -> dst [B, A].
hipError_t launch_u16_transpose(const uint16_t* src, uint16_t* dst, int64_t A, int64_t B, hipStream_t stream);
constexpr int64_t kU16TransposeMaxA = int64_t{65535} * 64;
constexpr int64_t kU16TransposeMaxB = int64_t{1} << 30;

// W4A16 GEMM y[M,N] = x[M,K] . dequant(qweight, scales, qzeros), groups of
// `group` rows (32, 64 or 128; K % 128 == 0). With a workspace of
// w4a16_gemm_workspace(M, N, K) bytes, K is split w4a16_gemm_splits ways
// when the tiles alone leave most CUs idle (fp32 partials, then a reduce
// kernel); a NULL workspace never splits.
int w4a16_gemm_splits(int64_t M, int64_t N, int64_t K);
size_t w4a16_gemm_workspace(int64_t M, int64_t N, int64_t K);
// bf16: x and y are bf16 (the weight is rounded once to bf16 instead of fp16).
// per_channel: scales / qzeros hold one row used for every group (the
// kernel runs with `group` rows per group, 128 for per-channel layers).
hipError_t launch_w4a16_gemm(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                             const int32_t* qzeros, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, int64_t group, bool per_channel, void* workspace,
                             bool bf16, hipStream_t stream);

// Largest token count the W4A16 GEMV takes (four 16-token MFMA tiles).
constexpr int64_t kGemvMaxM = 64;

// W4A16 GEMV launch plan: K is cut into `splits` slices across workgroups,
// each workgroup has `waves` wavefronts that share its K slice.
struct GemvPlan {
  int splits;
  int waves;  // wavefronts per workgroup (register-staged kernel)
  size_t workspace_bytes;
  bool lds;   // LDS-staged kernel (N % 32 == 0)
  int group;  // rows per group: 32, 64 or 128
  int strips_per_unit = 1;  // blocked GEMV: adjacent 32-output strips per workgroup
  bool per_channel = false; // one scale / zero-point row for all of K (group runs as 128)
};
GemvPlan plan_w4a16_gemv(int64_t M, int64_t N, int64_t K, int64_t group);

// Column-blocked weight layout for the decode GEMV (N % 128 == 0,
// K % 128 == 0): conversion from [K, N/8], plan and launch.
hipError_t launch_w4a16_block_weights(const int32_t* qweight, int32_t* blocked, int64_t N, int64_t K,
                                      hipStream_t stream);
GemvPlan plan_w4a16_gemv_blocked(int64_t M, int64_t N, int64_t K, int64_t group);
size_t w4a16_gemv_blocked_workspace(int64_t M, int64_t N, int64_t K, int64_t group);
hipError_t launch_w4a16_gemv_blocked(const uint16_t* x, const int32_t* blocked, const uint16_t* scales,
                                     const int32_t* qzeros, uint16_t* y, int64_t M, int64_t N, int64_t K,
                                     const GemvPlan& plan, void* workspace, bool bf16, hipStream_t stream);

hipError_t launch_w4a16_gemv(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                             const int32_t* qzeros, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, const GemvPlan& plan,
                             void* workspace, bool bf16, hipStream_t stream);

}  // namespace mq
