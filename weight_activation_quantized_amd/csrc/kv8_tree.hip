// Trees of drafted tokens over the paged e4m3 KV cache, for gfx950: which nodes
// see which and where they stand, and the cache's clean-up once some are kept.
#include "block8_launch.h"
#include "device_common.h"
#include "kv8_page.h"

namespace mq {
namespace {

// ---------------------------------------------------------------------------
// Masks and positions. Node j of a sequence has the parent parents[j] < j (in
// the sequence's own numbers; anything else: it hangs on the context). It sees
// itself and all above it:
//   seen(j) = {j} + seen(parent of j),  position(j) = context + |seen(j)| - 1
// A workgroup takes a sequence, a thread a node, which walks up and sets its row's
// bits in LDS. A word holds the three nodes above one, 10 bits each, so a step of
// the walk, one LDS read, goes up three. Bound by the launch, the loads and the walk:
// 8 nodes 2.1 us, 96 trees of 100-200 nodes 5.0 (one node a step, words to memory as
// they come: 6.4; 4 of 1000 nodes 21, 62).
// ---------------------------------------------------------------------------

constexpr int kNone = kKv8MaxTree - 1;  // (the last node is above no other)

// For trees of up to kNodes nodes.
template <int kNodes>
__global__ __launch_bounds__(kNodes) void kv8_tree_mask_kernel(const int32_t* __restrict__ parents,
                                                               const int32_t* __restrict__ cu,
                                                               const int32_t* __restrict__ lens,
                                                               int32_t* __restrict__ mask,
                                                               int32_t* __restrict__ positions, int tokens, int words,
                                                               int max_q_len) {
  constexpr int kWords = kNodes / 32, kPitch = kWords + 1;  // (of different banks)
  __shared__ uint32_t rows[kNodes * kPitch];
  __shared__ int up[kNodes];     // parents
  __shared__ int above[kNodes];  // three of them
  const int b = static_cast<int>(blockIdx.x), j = static_cast<int>(threadIdx.x);
  const int first = max(cu[b], 0), all = cu[b + 1] - cu[b];
  const int n = min(min(cu[b + 1], tokens) - first, max_q_len);  // (at most kNodes)
  const int start = lens[b] - all;
  int p = kNone;
  if (j < n) {
    p = parents[first + j];
    p = p >= 0 && p < j ? p : kNone;
  }
  up[j] = p;
  uint32_t* const row = rows + j * kPitch;
#pragma unroll
  for (int w = 0; w < kWords; ++w) row[w] = 0;
  __syncthreads();
  int q = p == kNone ? kNone : up[p], r = q == kNone ? kNone : up[q];
  above[j] = p | q << 10 | r << 20;
  __syncthreads();
  if (j < n) {
    auto see = [&](int at) { atomicOr(&row[at >> 5], 1u << (at & 31)); };  // (its own row: no read to wait for)
    see(j);
    int depth = 0;
    for (;;) {
      depth += (p != kNone) + (q != kNone) + (r != kNone);
      if (p != kNone) see(p);
      if (q != kNone) see(q);
      if (r == kNone) break;
      const int three = above[r];
      see(r);
      p = three & 1023;
      q = three >> 10 & 1023;
      r = three >> 20 & 1023;
    }
    positions[first + j] = start + depth;
  }
  __syncthreads();
  int32_t* const to = mask + static_cast<int64_t>(first) * words;
  for (int i = j; i < n * words; i += kNodes) {
    const int of = i / words, w = i - of * words;
    to[i] = w < kWords ? static_cast<int32_t>(rows[of * kPitch + w]) : 0;
  }
}

// ---------------------------------------------------------------------------
// Keeping a path: token i of the new ones becomes what node path[i] was, for
// i < kept. Nodes ascend, so path[i] >= i: sources lie in the same page as their
// places or behind it, and pages are done in order. Of each page (K and V apart,
// per head), with a = largest finite |code| * scale among the tokens that move
// into it,
//   s = max(s_old, smallest 2^e with a <= 448 2^e)
// moved codes become rne_e4m3(code * s_source / s), and where s grew all other
// codes of the page rne_e4m3(code * s_old / s). NaN codes stay NaN, and what a
// scale makes NaN or infinite arrives as the code of NaN.
//
// A workgroup owns one (layer, sequence, head, K or V): all codes that move into
// a page are in LDS before any of them is written. Bound by latency: lengths, the
// path's end, the page and its scale, and then for every 256 codes, a byte a lane,
// path, page and the code with its scale, which follow from each other and are waited
// for in each turn: five turns for nine tokens of 128 dimensions (8 layers of 16
// sequences, at most 9 tokens kept: 13.7 us; one wavefront for all of it 14.3-16,
// sources looked up ahead, still by bytes, 17).
// ---------------------------------------------------------------------------

constexpr int kKeepThreads = 256;

template <int D>
__global__ __launch_bounds__(kKeepThreads) void kv8_tree_keep_kernel(Kv8Cache c, const int32_t* __restrict__ path,
                                                                     const int32_t* __restrict__ kept, int width) {
  __shared__ uint8_t tile[128 * D];  // codes by token
  __shared__ float from[128];        // scale of each token's source; NaN: it does not move
  __shared__ int end;
  __shared__ float wmax[kKeepThreads / 64];
  unsigned at = blockIdx.x;
  const bool is_v = at & 1;
  at >>= 1;
  const int head = static_cast<int>(at % c.kv_heads);
  const int b = static_cast<int>(at / c.kv_heads);
  const size_t layer = blockIdx.y;
  const int n = c.cu[b + 1] - c.cu[b], start = c.lens[b] - n;
  const int most = min(min(kept[b], n), width);
  if (n <= 0 || start < 0 || most <= 0) return;
  const int32_t* const way = path + static_cast<size_t>(b) * width;
  if (threadIdx.x == 0) end = most;
  __syncthreads();
  for (int i = threadIdx.x; i < most; i += kKeepThreads)
    if (way[i] < i || way[i] >= n) atomicMin(&end, i);
  __syncthreads();
  const int count = end;
  const int32_t* const table = c.table + static_cast<size_t>(b) * c.table_width;
  auto page_of = [&](int pos) {  // -1: none
    const int slot = pos >> c.page_shift;
    const int id = slot < c.table_width ? table[slot] : -1;
    return id >= 0 && id < c.num_pages ? id : -1;
  };
  const size_t layer_unit = layer * c.num_pages * c.kv_heads + head;
  uint8_t* const codes = is_v ? c.v : c.k;
  float* const scales = is_v ? c.v_scales : c.k_scales;
  const int by_token = is_v ? 1 : D, by_dim = is_v ? c.page : 1;
  for (int pos0 = start & ~(c.page - 1); pos0 < start + count; pos0 += c.page) {
    const int lo = max(start - pos0, 0), hi = min(start + count - pos0, c.page);
    const int id = page_of(pos0);
    if (id < 0) continue;
    const size_t unit = layer_unit + static_cast<size_t>(id) * c.kv_heads;
    uint8_t* const out = codes + unit * c.page * D;
    const float old = scales[unit];
    float amax = 0.f;
    for (int i = threadIdx.x; i < (hi - lo) * D; i += kKeepThreads) {
      const int t = lo + i / D, d = i % D;
      const int node = way[pos0 + t - start];
      const int src = start + node, page = page_of(src);
      float s = __builtin_nanf("");
      if (page >= 0 && src != pos0 + t) {
        const size_t u = layer_unit + static_cast<size_t>(page) * c.kv_heads;
        s = scales[u];
        uint8_t code = codes[u * c.page * D + (src & (c.page - 1)) * by_token + d * by_dim];
        if (!(fabsf(s) < __builtin_inff())) {
          code = kNanCode;
          s = 1.f;
        }
        tile[t * D + d] = code;
        if ((code & 0x7f) != kNanCode) {
          const f32x2 v = __builtin_amdgcn_cvt_pk_f32_fp8(code, false);
          amax = fmaxf(amax, fabsf(v[0] * s));
        }
      }
      if (d == 0) from[t] = s;
    }
    amax = wave_max(amax);
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeepThreads / 64; ++i) amax = fmaxf(amax, wmax[i]);
    const float need = page_scale(amax);
    const bool grows = amax > 0.f && need > old;
    const float s = grows ? need : old;
    if (grows) {
      const float ratio = old / s;
      for (int i = threadIdx.x; i < c.page * D / 4; i += kKeepThreads) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(out) + i;
        *w = moved(*w, ratio);
      }
    }
    __syncthreads();  // every lane has read the old scale, and the other codes are in place
    if (threadIdx.x == 0) scales[unit] = s;
    for (int i = threadIdx.x; i < (hi - lo) * D; i += kKeepThreads) {
      const int t = lo + i / D, d = i % D;
      if (from[t] == from[t]) out[t * by_token + d * by_dim] = static_cast<uint8_t>(moved(tile[t * D + d], from[t] / s));
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_kv8_tree_mask(const int32_t* parents, const int32_t* cu, const int32_t* lens, int32_t* mask,
                                int32_t* positions, int tokens, int batch, int words, int max_q_len,
                                hipStream_t stream) {
  // the smallest workgroup that holds a tree (its rows take 1, 11 or 143 KB of LDS)
  const dim3 grid(static_cast<uint32_t>(batch));
  if (max_q_len <= 64)
    return launch_kernel(kv8_tree_mask_kernel<64>, grid, dim3(64), 0, stream, parents, cu, lens, mask, positions, tokens,
                         words, max_q_len);
  if (max_q_len <= 256)
    return launch_kernel(kv8_tree_mask_kernel<256>, grid, dim3(256), 0, stream, parents, cu, lens, mask, positions,
                         tokens, words, max_q_len);
  return launch_kernel(kv8_tree_mask_kernel<kKv8MaxTree>, grid, dim3(kKv8MaxTree), 0, stream, parents, cu, lens, mask,
                       positions, tokens, words, max_q_len);
}

hipError_t launch_kv8_tree_keep(const Kv8Cache& c, int layers, const int32_t* path, const int32_t* kept, int width,
                                hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(c.batch) * c.kv_heads * 2, static_cast<uint32_t>(layers));
  return c.head_dim == 128
             ? launch_kernel(kv8_tree_keep_kernel<128>, grid, dim3(kKeepThreads), 0, stream, c, path, kept, width)
             : launch_kernel(kv8_tree_keep_kernel<64>, grid, dim3(kKeepThreads), 0, stream, c, path, kept, width);
}

}  // namespace mq
