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
// All products and sums in binary64: a first child's test and the chains' are then
// exact (a product of two binary32 values has 48 bits), what is left to a later
// sibling is rounded by 2^-54 a term and its product once, and the drawn token does
// not depend on the order of a sum but within 2^-40 or so of a border.
//
// Whether a child is taken depends on single values of two rows: every node's
// are loaded at once, and one wavefront walks the tree by ballots. Only the last
// node's row is read whole, in pieces of 1024 values, one wavefront each, whose
// sums are kept; the piece of the drawn token is found among them and read again.
// Bound by HBM for many long rows (64 chains of 6 with the draft's probabilities,
// 128000 values: 19.0 us, 3.4 TB/s with the walk), else by the chain of dependent
// loads: offsets, nodes, their probabilities, the row, the piece (one tree of 8 over
// 32000: 8.6 us, without drafts 7.7).
#include "block8_launch.h"
#include "device_common.h"

namespace mq {
namespace {

constexpr int kPiece = 1024;        // values of a piece
constexpr int kPer = kPiece / 64;   // values of a lane
constexpr int kMaxKept = 256;       // pieces of a row whose sums fit a workgroup's LDS

// What the walk leaves of a sequence.
struct Walk {
  int32_t last, rejected;  // last node taken, rejected children of it
};

template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_f64(double x) {  // 0 where there is no source
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  const u32x2 r = {static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b[0]), kCtrl, kRows, 0xF, false)),
                   static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b[1]), kCtrl, kRows, 0xF, false))};
  return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  return __builtin_bit_cast(double, u32x2{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b[0]), lane)),
                                          static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b[1]), lane))});
}
__device__ __forceinline__ double wave_scan(double v) {  // of this lane and those before it
  v += dpp_f64<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v += dpp_f64<0x112, 0xF>(v);
  v += dpp_f64<0x114, 0xF>(v);
  v += dpp_f64<0x118, 0xF>(v);
  v += dpp_f64<0x142, 0xA>(v);  // row_bcast 15: rows 1 and 3
  v += dpp_f64<0x143, 0xC>(v);  // row_bcast 31: rows 2 and 3
  return v;
}
__device__ __forceinline__ double wave_total(double v) { return lane_f64(wave_scan(v), 63); }

__device__ __forceinline__ double mass(float p) { return p > 0.f ? static_cast<double>(p) : 0.; }

struct Sequence {
  int first, n;
};
__device__ __forceinline__ Sequence sequence_of(const VerifyArgs& a, int b) {
  const int first = max(a.cu[b], 0);
  return {first, min(min(a.cu[b + 1], a.tokens) - first, a.max_q_len)};
}

// The nodes of a sequence, and the rejected tokens of the last one taken.
struct Nodes {
  int32_t token[kKv8MaxTree], parent[kKv8MaxTree], gone[kKv8MaxTree];
  float p[kKv8MaxTree], q[kKv8MaxTree], u[kKv8MaxTree];
  Walk walk;
};

// Walks the tree of sequence b, by the whole workgroup; `tells`: the one that
// writes kept and path.
__device__ __forceinline__ Walk walk_tree(const VerifyArgs& a, Nodes& s, int b, const Sequence& seq, bool tells) {
  const int first = seq.first, n = seq.n;
  int32_t* const path = a.path + static_cast<int64_t>(b) * a.max_q_len;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int up = a.parents ? a.parents[first + j] : j - 1;
    const int x = a.token[first + j];
    const bool real = up >= 0 && up < j;
    const bool known = real && x >= 0 && x < a.vocab;
    const int64_t at = static_cast<int64_t>(first + (real ? up : 0)) * a.vocab + (known ? x : 0);
    s.token[j] = x;
    s.parent[j] = real ? up : -1;
    s.p[j] = known ? a.probs[at] : 0.f;
    s.q[j] = known && a.draft ? fmaxf(a.draft[at], 0.f) : 1.f;  // (NaN: 0)
    s.u[j] = a.uniform[first + j];
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int last = 0, taken = 1, rejected = 0;
    double left = 1.;
    if (tells && lane == 0) path[0] = 0;
    for (int j0 = 0; j0 < n; j0 += 64) {
      const int j = j0 + lane;
      const int up = j < n ? s.parent[j] : -1;
      uint64_t mine = __ballot(j < n && up == last);
      while (mine) {
        const int child = j0 + __builtin_ctzll(mine);
        const int x = s.token[child];
        bool again = false;  // the token of a rejected sibling
        for (int r0 = 0; r0 < rejected; r0 += 64) again |= __any(r0 + lane < rejected && s.gone[r0 + lane] == x);
        const double p = again ? 0. : mass(s.p[child]);
        // (what is left may have fallen below 0 by the row's rounding: a token of p = 0 stays out)
        const bool yes = static_cast<double>(s.u[child]) * (a.draft ? static_cast<double>(s.q[child]) : fmax(left, 0.)) < p;
        if (yes) {
          if (tells && lane == 0) path[taken] = child;
          ++taken;
          last = child;
          left = 1.;
          rejected = 0;
          mine = __ballot(j < n && up == last);
        } else {
          left -= p;
          s.gone[rejected] = x;  // (every lane the same)
          ++rejected;
          mine &= mine - 1;
        }
      }
    }
    if (lane == 0) {
      s.walk = {last, rejected};
      if (tells) a.kept[b] = taken;
    }
    if (tells)
      for (int i = taken + lane; i < a.max_q_len; i += 64) path[i] = -1;
  }
  __syncthreads();
  return s.walk;
}

// A sequence without rows.
__device__ __forceinline__ void tell_empty(const VerifyArgs& a, int b) {
  for (int i = threadIdx.x; i < a.max_q_len; i += blockDim.x) a.path[static_cast<int64_t>(b) * a.max_q_len + i] = -1;
  if (threadIdx.x == 0) {
    a.kept[b] = 0;
    a.next[b] = -1;
  }
}

// The row that is drawn from.
struct Row {
  const float* p;
  const float* q;  // NULL: nothing to be taken off
  int vocab;
  __device__ __forceinline__ Row(const VerifyArgs& a, const Sequence& seq, const Walk& w) : vocab(a.vocab) {
    const int64_t at = static_cast<int64_t>(seq.first + w.last) * a.vocab;
    p = a.probs + at;
    q = a.draft && w.rejected ? a.draft + at : nullptr;
  }
};
__device__ __forceinline__ double rest_of(double p, float q) {
  const double d = p - mass(q);
  return d > 0. ? d : 0.;
}

// Sums of piece z, by one wavefront: the rest's, without the `rejected` tokens of
// `gone`, and the whole row's. kVec: rows are 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ void piece_sums(const Row& row, const int32_t* gone, int rejected, int z, double& rest,
                                           double& whole) {
  const int lane = threadIdx.x & 63, v0 = z * kPiece;
  float p[kPer], q[kPer];
  int v[kPer];
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const int at = v0 + 256 * i + 4 * lane;
      const bool in = at < row.vocab;
      f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
      if (in) x = *reinterpret_cast<const f32x4*>(row.p + at);
      if (in && row.q) y = *reinterpret_cast<const f32x4*>(row.q + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[4 * i + e] = at + e;
        p[4 * i + e] = x[e];
        q[4 * i + e] = y[e];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = v0 + 64 * i + lane;
      p[i] = q[i] = 0.f;
      if (v[i] < row.vocab) p[i] = row.p[v[i]];
      if (v[i] < row.vocab && row.q) q[i] = row.q[v[i]];
    }
  }
  double r[kPer];
  whole = 0.;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const double m = mass(p[i]);
    whole += m;
    r[i] = row.q ? rest_of(m, q[i]) : m;
  }
  if (gone)
    for (int e = 0; e < rejected; ++e) {
      const int x = gone[e];
      if (x < v0 || x >= v0 + kPiece) continue;
#pragma unroll
      for (int i = 0; i < kPer; ++i) r[i] = v[i] == x ? 0. : r[i];
    }
  rest = 0.;
#pragma unroll
  for (int i = 0; i < kPer; ++i) rest += r[i];
  rest = wave_total(rest);
  whole = wave_total(whole);
}

// What the token is looked for with: by each wavefront alike, from the pieces'
// sums, (rest, whole) one after the other.
struct Found {
  int piece;  // -1: the row has no mass
  bool left;  // the rest has some
  double limit, before;
};
__device__ __forceinline__ Found find_piece(const double* sums, int pieces, float uniform) {
  const int lane = threadIdx.x & 63;
  double total[2] = {0., 0.};
  for (int z0 = 0; z0 < pieces; z0 += 64) {
    const bool in = z0 + lane < pieces;
    total[0] += wave_total(in ? sums[2 * (z0 + lane)] : 0.);
    total[1] += wave_total(in ? sums[2 * (z0 + lane) + 1] : 0.);
  }
  Found f = {-1, total[0] > 0., 0., 0.};
  const double all = f.left ? total[0] : total[1];
  if (!(all > 0.)) return f;
  f.limit = static_cast<double>(uniform) * all;
  // The first piece whose end passes the limit, else the last one with any mass.
  int some = 0;
  double sum = 0., before_some = 0.;
  for (int z0 = 0; z0 < pieces && f.piece < 0; z0 += 64) {
    const double v = z0 + lane < pieces ? sums[2 * (z0 + lane) + (f.left ? 0 : 1)] : 0.;
    const double scan = sum + wave_scan(v);
    const uint64_t past = __ballot(v > 0. && scan > f.limit), any = __ballot(v > 0.);
    if (any) {
      const int at = 63 - __builtin_clzll(any);
      some = z0 + at;
      before_some = lane_f64(scan - v, at);
    }
    if (past) {
      const int at = __builtin_ctzll(past);
      f.piece = z0 + at;
      f.before = lane_f64(scan - v, at);
    }
    sum = lane_f64(scan, 63);
  }
  if (f.piece < 0) {
    f.piece = some;
    f.before = before_some;
  }
  return f;
}

// The token, by the first wavefront: 16 values side by side in a lane.
__device__ __forceinline__ void pick(const VerifyArgs& a, int b, const Row& row, const int32_t* gone, int rejected,
                                     const Found& f) {
  const int lane = threadIdx.x & 63;
  const int v0 = f.piece * kPiece + lane * kPer;
  const bool off = row.q && f.left;
  float p[kPer], q[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] = q[i] = 0.f;
    if (v0 + i < row.vocab) p[i] = row.p[v0 + i];
    if (v0 + i < row.vocab && off) q[i] = row.q[v0 + i];
  }
  double r[kPer], mine = 0.;
#pragma unroll
  for (int i = 0; i < kPer; ++i) r[i] = off ? rest_of(mass(p[i]), q[i]) : mass(p[i]);
  if (gone && f.left)
    for (int e = 0; e < rejected; ++e) {
      const int x = gone[e] - v0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) r[i] = x == i ? 0. : r[i];
    }
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += r[i];
  double cum = f.before + (wave_scan(mine) - mine);
  int found = -1, some = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cum += r[i];
    if (r[i] > 0.) {
      some = v0 + i;
      if (cum > f.limit && found < 0) found = v0 + i;
    }
  }
  const uint64_t hits = __ballot(found >= 0), any = __ballot(some >= 0);
  int token = -1;
  if (hits) {
    token = __builtin_amdgcn_readlane(found, __builtin_ctzll(hits));
  } else if (any) {
    token = __builtin_amdgcn_readlane(some, 63 - __builtin_clzll(any));
  }
  if (lane == 0) a.next[b] = token;
}

// One workgroup per sequence, all of it.
template <bool kVec>
__global__ __launch_bounds__(1024) void draft_verify_kernel(VerifyArgs a, int pieces) {
  __shared__ Nodes nodes;
  __shared__ double sums[2 * kMaxKept];
  const int b = static_cast<int>(blockIdx.x);
  const Sequence seq = sequence_of(a, b);
  if (seq.n <= 0) return tell_empty(a, b);
  const Walk walk = walk_tree(a, nodes, b, seq, true);
  const Row row(a, seq, walk);
  const int32_t* const gone = a.draft ? nullptr : nodes.gone;
  for (int z = threadIdx.x >> 6; z < pieces; z += 16) {
    double rest, whole;
    piece_sums<kVec>(row, gone, walk.rejected, z, rest, whole);
    if ((threadIdx.x & 63) == 0) {
      sums[2 * z] = rest;
      sums[2 * z + 1] = whole;
    }
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const Found f = find_piece(sums, pieces, nodes.u[0]);
  if (f.piece >= 0) return pick(a, b, row, gone, walk.rejected, f);
  if (threadIdx.x == 0) a.next[b] = -1;
}

// Several workgroups per sequence, each walks for itself and leaves its pieces'
// sums; the token by a second launch.
template <bool kVec>
__global__ __launch_bounds__(256) void draft_sums_kernel(VerifyArgs a, int pieces) {
  __shared__ Nodes nodes;
  const int b = static_cast<int>(blockIdx.y), part = static_cast<int>(blockIdx.x), parts = static_cast<int>(gridDim.x);
  const Sequence seq = sequence_of(a, b);
  if (seq.n <= 0) {
    if (part == 0) tell_empty(a, b);
    return;
  }
  const Walk walk = walk_tree(a, nodes, b, seq, part == 0);
  if (part == 0) {
    if (threadIdx.x == 0) reinterpret_cast<Walk*>(a.walks)[b] = walk;
    int32_t* const list = a.lists + static_cast<int64_t>(b) * a.max_q_len;
    for (int i = threadIdx.x; i < walk.rejected; i += 256) list[i] = nodes.gone[i];
  }
  const Row row(a, seq, walk);
  for (int z = 4 * part + (static_cast<int>(threadIdx.x) >> 6); z < pieces; z += 4 * parts) {
    double rest, whole;
    piece_sums<kVec>(row, a.draft ? nullptr : nodes.gone, walk.rejected, z, rest, whole);
    if ((threadIdx.x & 63) == 0) {
      double* const to = a.sums + 2 * (static_cast<int64_t>(b) * pieces + z);
      to[0] = rest;
      to[1] = whole;
    }
  }
}

__global__ __launch_bounds__(64) void draft_pick_kernel(VerifyArgs a, int pieces) {
  const int b = static_cast<int>(blockIdx.x);
  const Sequence seq = sequence_of(a, b);
  if (seq.n <= 0) return;
  const Walk walk = reinterpret_cast<const Walk*>(a.walks)[b];
  const Found f = find_piece(a.sums + 2 * static_cast<int64_t>(b) * pieces, pieces, a.uniform[seq.first]);
  if (f.piece >= 0)
    return pick(a, b, Row(a, seq, walk), a.draft ? nullptr : a.lists + static_cast<int64_t>(b) * a.max_q_len, walk.rejected, f);
  if (threadIdx.x == 0) a.next[b] = -1;
}

int pieces_of(int vocab) { return (vocab + kPiece - 1) / kPiece; }

// One workgroup for a sequence where its 16 wavefronts have a piece each, or where
// there are sequences for all compute units; otherwise workgroups of four
// wavefronts, as many as make 512, and a second launch (both measured, in us: one
// sequence without drafts, 16000 values, 7.0, with two launches 7.6; 32000 7.7, in
// one 9.0; a tree of 8 over 16000 8.1, in two 8.4; over 32000 8.6, in one 10.4; 64
// chains of 6 over 128000 with the draft's 19.0, in one 25.8, with 256 or 2048
// workgroups 19.9 and 20.3; 256 of 2 over 128000 31.7, in two launches 40.7).
constexpr int kOwnPieces = 16, kManyRows = 256, kWorkgroups = 512;
bool in_one(int batch, int vocab) { return pieces_of(vocab) <= (batch >= kManyRows ? kMaxKept : kOwnPieces); }

template <bool kVec>
hipError_t launch(const VerifyArgs& a, int batch, hipStream_t stream) {
  const int pieces = pieces_of(a.vocab);
  const uint32_t rows = static_cast<uint32_t>(batch);
  if (in_one(batch, a.vocab))
    return launch_kernel(draft_verify_kernel<kVec>, dim3(rows), dim3(1024), 0, stream, a, pieces);
  const int most = (pieces + 3) / 4, want = (kWorkgroups + batch - 1) / batch;
  const hipError_t e = launch_kernel(draft_sums_kernel<kVec>, dim3(static_cast<uint32_t>(want < most ? want : most), rows),
                                     dim3(256), 0, stream, a, pieces);
  if (e != hipSuccess) return e;
  return launch_kernel(draft_pick_kernel, dim3(rows), dim3(64), 0, stream, a, pieces);
}

}  // namespace

size_t verify_workspace(int batch, int vocab, int max_q_len) {
  if (in_one(batch, vocab)) return 0;
  return static_cast<size_t>(batch) * (16 * static_cast<size_t>(pieces_of(vocab)) + sizeof(Walk) + 4 * static_cast<size_t>(max_q_len));
}

hipError_t launch_draft_verify(VerifyArgs a, int batch, void* workspace, hipStream_t stream) {
  a.sums = static_cast<double*>(workspace);
  a.walks = a.sums + static_cast<size_t>(batch) * pieces_of(a.vocab) * 2;
  a.lists = static_cast<int32_t*>(static_cast<void*>(static_cast<Walk*>(a.walks) + batch));
  const bool vec = a.vocab % 4 == 0 && reinterpret_cast<uintptr_t>(a.probs) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.draft) % 16 == 0;
  return vec ? launch<true>(a, batch, stream) : launch<false>(a, batch, stream);
}

}  // namespace mq
