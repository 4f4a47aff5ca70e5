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

// The same with q and k [tokens, heads, head_dim] normed per head where weights
// are given and rotated: the cosines and sines of position p are row p of
// cos_sin, pairs lie rot / 2 apart or next to each other.
struct Kv8Turn {
  const uint16_t* q;
  uint16_t* q_out;  // q itself (of the same stride) or apart from everything
  int64_t q_stride, q_out_stride;
  const float* cos_sin;        // [max_pos, rot]: rot / 2 cosines, rot / 2 sines
  const int32_t* positions;    // [tokens]; NULL: a token's place in its sequence
  const uint16_t* q_weight;    // [head_dim] both, or NULL both: no norm
  const uint16_t* k_weight;
  double eps;
  int q_heads, max_pos, rot;  // rot: a multiple of 16, at most head_dim
  bool next;
  // by plan_kv8_turn: workgroups of the queries take `tile` tokens and `heads_of` heads,
  // `tiles` and `parts` of them a sequence
  int tile, heads_of, tiles, parts;
  uint32_t share;  // of all workgroups, by the launcher
};
Kv8Turn plan_kv8_turn(const Kv8Cache& c, Kv8Turn t);
int64_t kv8_rope_append_blocks(const Kv8Cache& c, const Kv8Turn& t);  // workgroups of the launch
hipError_t launch_kv8_rope_append(const Kv8Cache& c, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                  int64_t v_stride, const Kv8Turn& turning, bool bf16, hipStream_t stream);

// out [tokens, q_heads, head_dim] = causal attention of q over the cache. With
// plan.splits > 1 every split of the keys leaves its part in the workspace and
// a second kernel joins them.
struct Kv8Plan {
  bool decode;  // the rows of one kv head fit a few tiles of 16: the streaming form
  int waves;    // wavefronts of a workgroup
  int splits;
  int64_t prompt_blocks;  // workgroups of the other form (under 2^29 within the entry's limits)
  int least;              // (of trees) tiles of keys that such a workgroup takes at least
  size_t workspace_bytes;
};
Kv8Plan plan_kv8_attention(const Kv8Cache& c, int q_heads);
hipError_t launch_kv8_attention(const Kv8Cache& c, const uint16_t* q, int64_t q_stride, uint16_t* out, int q_heads,
                                float softmax_scale, const Kv8Plan& plan, void* workspace, bool bf16,
                                hipStream_t stream);

// Attention of drafted tokens: a row sees every token before the new ones, and of
// those the ones that its words name (bit j of [tokens, words]: new token j).
struct Kv8Tree {
  const int32_t* mask;
  int words;
};
constexpr int kKv8MaxTree = 1024;  // new tokens of a sequence
Kv8Plan plan_kv8_tree_attention(const Kv8Cache& c, int q_heads);
hipError_t launch_kv8_tree_attention(const Kv8Cache& c, const uint16_t* q, int64_t q_stride, const Kv8Tree& tree,
                                     uint16_t* out, int q_heads, float softmax_scale, const Kv8Plan& plan,
                                     void* workspace, bool bf16, hipStream_t stream);

// Those words and the tokens' positions, from each node's parent.
hipError_t launch_kv8_tree_mask(const int32_t* parents, const int32_t* cu, const int32_t* lens, int32_t* mask,
                                int32_t* positions, int tokens, int batch, int words, int max_q_len,
                                hipStream_t stream);

// New token i becomes what new token path[b, i] was, for i < kept[b], in each of
// `layers` caches that lie one behind the other; path [batch, width].
hipError_t launch_kv8_tree_keep(const Kv8Cache& c, int layers, const int32_t* path, const int32_t* kept, int width,
                                hipStream_t stream);

// Drafted tokens against the target's probabilities.
struct VerifyArgs {
  const float* probs;      // [tokens, vocab]
  const float* draft;      // the same, or NULL
  const int32_t* token;    // [tokens]
  const int32_t* parents;  // [tokens], or NULL: chains
  const float* uniform;    // [tokens]
  const int32_t* cu;       // [batch + 1]
  int32_t *kept, *path, *next;  // [batch], [batch, max_q_len], [batch]
  int tokens, vocab, max_q_len;
  // in the workspace, set by the launcher
  double* sums;
  void* walks;
  int32_t* lists;
};
size_t verify_workspace(int batch, int vocab, int max_q_len);
hipError_t launch_draft_verify(VerifyArgs a, int batch, void* workspace, hipStream_t stream);

}  // namespace mq
