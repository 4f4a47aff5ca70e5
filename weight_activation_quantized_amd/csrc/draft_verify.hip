// Verification of drafted tokens against the target's probabilities, for gfx950.
//
// A sequence's node 0 is its last certain token, row j of `probs` the target's
// distribution of the token that follows node j. From node 0 on, the children of
// the last node taken are tried in order; child c, the token x, is taken iff
//   trees:                      u_c (1 - sum of p(x') of the siblings rejected before it) < p(x)
//   chains drawn from q:        u_c q(x) < p(x)
// (p = 0 for the token of a rejected sibling). The token after the last node
// taken is drawn from what the rejections leave of its row: p without the
// rejected tokens, or max(0, p - q); from p where nothing was rejected or
// nothing is left. With r that rest, it is the smallest v with
//   sum_{w <= v} r(w) > u_0 sum_w r(w)
// All products and sums in binary64: tests of binary32 values are then exact, and
// the drawn token does not depend on the order of a sum but within 2^-40 or so
// of a border.
//
// Whether a child is taken depends on single values of two rows: every node's
// are loaded at once, and one wavefront walks the tree by ballots. Only the last
// node's row is read whole, by as many workgroups as it has pieces of 4096; each
// walks for itself and leaves its sums, and a second launch (one workgroup per
// sequence) finds the piece, then the token.
#include "block8_launch.h"
#include "device_common.h"

namespace mq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = kVerifyPiece / kThreads;  // values per thread

// What the walk leaves of a sequence, in the workspace.
struct Walk {
  int32_t last, rejected;  // last node taken, rejected children of it
};

__device__ __forceinline__ double wave_scan(double v) {  // of this lane and those before it
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double below = __shfl_up(v, d, kWave);
    v += lane >= d ? below : 0.;
  }
  return v;
}

__device__ __forceinline__ double mass(float p) { return p > 0.f ? static_cast<double>(p) : 0.; }

// The rest r of thread's values v0 + kThreads i (coalesced) or v0 + i.
struct Row {
  const float* p;
  const float* q;  // NULL: none to be taken off
  int vocab;
  __device__ __forceinline__ double rest(int v) const {
    if (v >= vocab) return 0.;
    const double a = mass(p[v]);
    if (!q) return a;
    const double d = a - static_cast<double>(q[v]);
    return d > 0. ? d : 0.;
  }
};

__global__ __launch_bounds__(kThreads) void draft_walk_kernel(VerifyArgs a) {
  __shared__ int32_t token[kKv8MaxTree], parent[kKv8MaxTree], gone[kKv8MaxTree];
  __shared__ float pv[kKv8MaxTree], qv[kKv8MaxTree], uv[kKv8MaxTree];
  __shared__ int s_last, s_rejected;
  __shared__ double sums[2][kThreads / 64];
  const int b = static_cast<int>(blockIdx.y), piece = static_cast<int>(blockIdx.x);
  const int first = max(a.cu[b], 0), n = min(min(a.cu[b + 1], a.tokens) - first, a.max_q_len);
  int32_t* const path = a.path + static_cast<int64_t>(b) * a.max_q_len;
  if (n <= 0) {
    if (piece == 0) {
      for (int i = threadIdx.x; i < a.max_q_len; i += kThreads) path[i] = -1;
      if (threadIdx.x == 0) {
        a.kept[b] = 0;
        a.next[b] = -1;
      }
    }
    return;
  }
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int up = a.parents ? a.parents[first + j] : j - 1;
    const int x = a.token[first + j];
    const bool real = up >= 0 && up < j;
    const bool known = real && x >= 0 && x < a.vocab;
    const int64_t at = static_cast<int64_t>(first + (real ? up : 0)) * a.vocab + (known ? x : 0);
    token[j] = x;
    parent[j] = real ? up : -1;
    pv[j] = known ? a.probs[at] : 0.f;
    qv[j] = known && a.draft ? a.draft[at] : 1.f;
    uv[j] = a.uniform[first + j];
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int last = 0, taken = 1, rejected = 0;
    double left = 1.;
    if (piece == 0 && lane == 0) path[0] = 0;
    for (int j0 = 0; j0 < n; j0 += 64) {
      const int j = j0 + lane;
      const int up = j < n ? parent[j] : -1;
      uint64_t mine = __ballot(j < n && up == last);
      while (mine) {
        const int child = j0 + __builtin_ctzll(mine);
        const int x = token[child];
        bool again = false;  // the token of a rejected sibling
        for (int r0 = 0; r0 < rejected; r0 += 64) again |= __any(r0 + lane < rejected && gone[r0 + lane] == x);
        const double p = again ? 0. : mass(pv[child]);
        const bool yes = static_cast<double>(uv[child]) * (a.draft ? static_cast<double>(qv[child]) : left) < p;
        if (yes) {
          if (piece == 0 && lane == 0) path[taken] = child;
          ++taken;
          last = child;
          left = 1.;
          rejected = 0;
          mine = __ballot(j < n && up == last);
        } else {
          left -= p;
          gone[rejected] = x;  // (every lane the same)
          ++rejected;
          mine &= mine - 1;
        }
      }
    }
    if (lane == 0) {
      s_last = last;
      s_rejected = rejected;
      if (piece == 0) a.kept[b] = taken;
    }
    if (piece == 0)
      for (int i = taken + lane; i < a.max_q_len; i += 64) path[i] = -1;
  }
  __syncthreads();
  const int last = s_last, rejected = s_rejected;
  const int64_t at = static_cast<int64_t>(first + last) * a.vocab;
  const Row row = {a.probs + at, a.draft && rejected ? a.draft + at : nullptr, a.vocab};
  int32_t* const list = a.lists + static_cast<int64_t>(b) * a.max_q_len;
  if (piece == 0) {
    if (threadIdx.x == 0) reinterpret_cast<Walk*>(a.walks)[b] = {last, rejected};
    for (int i = threadIdx.x; i < rejected; i += kThreads) list[i] = gone[i];
  }
  double rest = 0., whole = 0.;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = piece * kVerifyPiece + i * kThreads + static_cast<int>(threadIdx.x);
    double r = row.rest(v);
    whole += row.q ? (v < a.vocab ? mass(row.p[v]) : 0.) : r;
    if (!a.draft)
      for (int e = 0; e < rejected; ++e) r = gone[e] == v ? 0. : r;
    rest += r;
  }
  rest = __shfl(wave_scan(rest), 63, kWave);
  whole = __shfl(wave_scan(whole), 63, kWave);
  if ((threadIdx.x & 63) == 63) {
    sums[0][threadIdx.x >> 6] = rest;
    sums[1][threadIdx.x >> 6] = whole;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double* const to = a.sums + 2 * (static_cast<int64_t>(b) * gridDim.x + piece);
    to[0] = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
    to[1] = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
  }
}

__global__ __launch_bounds__(kThreads) void draft_pick_kernel(VerifyArgs a, int pieces) {
  __shared__ double sums[kThreads / 64];
  __shared__ int s_first, s_any;
  const int b = static_cast<int>(blockIdx.x);
  const int first = max(a.cu[b], 0), n = min(min(a.cu[b + 1], a.tokens) - first, a.max_q_len);
  if (n <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Walk walk = reinterpret_cast<const Walk*>(a.walks)[b];
  const double* const parts = a.sums + 2 * static_cast<int64_t>(b) * pieces;
  // Every wavefront adds the pieces' sums up, 64 at a time, in the same order.
  auto total_of = [&](int which) {
    double sum = 0.;
    for (int z0 = 0; z0 < pieces; z0 += 64) {
      const double v = z0 + lane < pieces ? parts[2 * (z0 + lane) + which] : 0.;
      sum += __shfl(wave_scan(v), 63, kWave);
    }
    return sum;
  };
  double total = total_of(0);
  const bool left = total > 0.;
  if (!left) total = total_of(1);
  if (!(total > 0.)) {  // a row without any mass
    if (threadIdx.x == 0) a.next[b] = -1;
    return;
  }
  const double limit = static_cast<double>(a.uniform[first]) * total;
  // The first piece whose end passes the limit, else the last one with any mass.
  int piece = -1, some = 0;
  double before = 0., sum = 0., before_some = 0.;
  for (int z0 = 0; z0 < pieces && piece < 0; z0 += 64) {
    const double v = z0 + lane < pieces ? parts[2 * (z0 + lane) + (left ? 0 : 1)] : 0.;
    const double scan = sum + wave_scan(v);
    const uint64_t past = __ballot(v > 0. && scan > limit), any = __ballot(v > 0.);
    if (any) {
      const int at = 63 - __builtin_clzll(any);
      some = z0 + at;
      before_some = __shfl(scan - v, at, kWave);
    }
    if (past) {
      const int at = __builtin_ctzll(past);
      piece = z0 + at;
      before = __shfl(scan - v, at, kWave);
    }
    sum = __shfl(scan, 63, kWave);
  }
  if (piece < 0) {
    piece = some;
    before = before_some;
  }
  // This thread's values lie side by side.
  const int64_t at = static_cast<int64_t>(first + walk.last) * a.vocab;
  const Row row = {a.probs + at, a.draft && walk.rejected && left ? a.draft + at : nullptr, a.vocab};
  const int32_t* const list = a.lists + static_cast<int64_t>(b) * a.max_q_len;
  const int v0 = piece * kVerifyPiece + static_cast<int>(threadIdx.x) * kPer;
  double r[kPer], mine = 0.;
#pragma unroll
  for (int i = 0; i < kPer; ++i) r[i] = row.rest(v0 + i);
  if (!a.draft && left)
    for (int e = 0; e < walk.rejected; ++e) {
      const int x = list[e] - v0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) r[i] = x == i ? 0. : r[i];
    }
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += r[i];
  const double scan = wave_scan(mine);
  if (lane == 63) sums[wave] = scan;
  if (threadIdx.x == 0) {
    s_first = 0x7fffffff;
    s_any = -1;
  }
  __syncthreads();
  double cum = before + (scan - mine);
  for (int w = 0; w < wave; ++w) cum += sums[w];
  int found = 0x7fffffff, any = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cum += r[i];
    if (r[i] > 0.) {
      any = v0 + i;
      if (cum > limit && found == 0x7fffffff) found = v0 + i;
    }
  }
  if (found != 0x7fffffff) atomicMin(&s_first, found);
  if (any >= 0) atomicMax(&s_any, any);
  __syncthreads();
  if (threadIdx.x == 0) a.next[b] = s_first != 0x7fffffff ? s_first : s_any;
}

}  // namespace

int verify_pieces(int vocab) { return (vocab + kVerifyPiece - 1) / kVerifyPiece; }

size_t verify_workspace(int batch, int vocab, int max_q_len) {
  return static_cast<size_t>(batch) * (16 * verify_pieces(vocab) + sizeof(Walk) + 4 * static_cast<size_t>(max_q_len));
}

hipError_t launch_draft_verify(VerifyArgs a, int batch, void* workspace, hipStream_t stream) {
  const int pieces = verify_pieces(a.vocab);
  a.sums = static_cast<double*>(workspace);
  a.walks = a.sums + static_cast<size_t>(batch) * pieces * 2;
  a.lists = static_cast<int32_t*>(static_cast<void*>(static_cast<Walk*>(a.walks) + batch));
  const hipError_t e = launch_kernel(draft_walk_kernel, dim3(static_cast<uint32_t>(pieces), static_cast<uint32_t>(batch)),
                                     dim3(kThreads), 0, stream, a);
  if (e != hipSuccess) return e;
  return launch_kernel(draft_pick_kernel, dim3(static_cast<uint32_t>(batch)), dim3(kThreads), 0, stream, a, pieces);
}

}  // namespace mq
