// C ABI of libmq: argument validation (host only, before any HIP call),
// status strings, thread-local error detail, and dispatch to the kernels.
// The operations and their sources are documented in include/mq.h.
#include "mq.h"

#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "block8_launch.h"
#include "launch.h"

namespace {

thread_local char g_last_error[512] = "";

mq_status fail(mq_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

mq_status ok() {
  g_last_error[0] = '\0';
  return MQ_OK;
}

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxK = int64_t{1} << 20;
constexpr int64_t kMaxKInt8 = 133136;            // largest multiple of 16 with 127 * 127 * K < 2^31
constexpr int64_t kMaxElems = int64_t{1} << 40;  // bound on M*N, M*K, K*N
constexpr int64_t kMaxN4 = int64_t{1} << 27;     // W4A16 N (32-bit lane offsets)

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};

bool overlap(const Range& a, const Range& b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Every output must be disjoint from every input and from the other outputs.
template <size_t NI, size_t NO>
mq_status check_alias(const Range (&in)[NI], const Range (&out)[NO]) {
  for (size_t o = 0; o < NO; ++o) {
    for (size_t i = 0; i < NI; ++i)
      if (overlap(out[o], in[i]))
        return fail(MQ_ERR_ALIAS, "output %s overlaps input %s", out[o].name, in[i].name);
    for (size_t p = o + 1; p < NO; ++p)
      if (overlap(out[o], out[p]))
        return fail(MQ_ERR_ALIAS, "output %s overlaps output %s", out[o].name, out[p].name);
  }
  return MQ_OK;
}

mq_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(MQ_ERR_HIP, "%s: %s (%s)", what, hipGetErrorName(e), hipGetErrorString(e));
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// A tensor pointer may be NULL only when the tensor has no elements (an
// empty torch tensor reports a NULL data pointer).
mq_status need(const void* p, int64_t elems, const char* name) {
  if (p == nullptr && elems > 0) return fail(MQ_ERR_NULL, "%s is NULL", name);
  return MQ_OK;
}

#define MQ_TRY(expr)                  \
  do {                                \
    const mq_status st_ = (expr);     \
    if (st_ != MQ_OK) return st_;     \
  } while (0)

mq_status check_mk(int64_t M, int64_t K, int64_t k_min, int64_t k_max, int64_t k_mult) {
  if (M < 0 || M > kMaxDim) return fail(MQ_ERR_SHAPE, "M=%lld out of range", (long long)M);
  if (K < k_min || K > k_max) return fail(MQ_ERR_SHAPE, "K=%lld out of [%lld, %lld]", (long long)K,
                                          (long long)k_min, (long long)k_max);
  if (K % k_mult) return fail(MQ_ERR_SHAPE, "K=%lld is not a multiple of %lld", (long long)K, (long long)k_mult);
  if (M * K > kMaxElems) return fail(MQ_ERR_SHAPE, "M*K too large");
  return MQ_OK;
}

// group -1: one scale and zero point per output column over all of K
// (per-channel); the kernels run it as groups of 128 rows that all read the
// one parameter row.
bool w4a16_group_ok(int64_t group) { return group == 32 || group == 64 || group == 128 || group == -1; }
int64_t kernel_group(int64_t group) { return group == -1 ? 128 : group; }
size_t group_rows(int64_t K, int64_t group) { return group == -1 ? 1 : static_cast<size_t>(K / group); }

mq_status check_w4a16(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                      const int32_t* qzeros, uint16_t* y, int64_t M, int64_t N, int64_t K, int64_t group) {
  if (!w4a16_group_ok(group))
    return fail(MQ_ERR_UNSUPPORTED, "group=%lld (32, 64, 128 and -1 = per-channel are provided)", (long long)group);
  MQ_TRY(check_mk(M, K, 128, kMaxK, 128));
  if (N < 8 || N > kMaxN4 || N % 8)
    return fail(MQ_ERR_SHAPE, "N=%lld must be a multiple of 8 in [8, 2^27]", (long long)N);
  if (M * N > kMaxElems || K * N > kMaxElems) return fail(MQ_ERR_SHAPE, "problem too large");
  MQ_TRY(need(x, M * K, "x"));
  MQ_TRY(need(qweight, K * N, "qweight"));
  MQ_TRY(need(scales, N, "scales"));
  MQ_TRY(need(qzeros, N, "qzeros"));
  MQ_TRY(need(y, M * N, "y"));
  if (!aligned(x, 16) || !aligned(scales, 16) || !aligned(y, 16))
    return fail(MQ_ERR_ALIGN, "x, scales and y must be 16-byte aligned");
  if (!aligned(qweight, 4) || !aligned(qzeros, 4))
    return fail(MQ_ERR_ALIGN, "qweight and qzeros must be 4-byte aligned");
  const size_t G = group_rows(K, group);
  const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"},
                      {qweight, static_cast<size_t>(K * (N / 8)) * 4, "qweight"},
                      {scales, G * static_cast<size_t>(N) * 2, "scales"},
                      {qzeros, G * static_cast<size_t>(N / 8) * 4, "qzeros"}};
  const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}};
  return check_alias(in, out);
}

mq_status check_w8a8(const int8_t* xq, const int8_t* wq, const void* out, size_t out_elem,
                     int64_t M, int64_t N, int64_t K) {
  mq_status s = check_mk(M, K, 16, kMaxKInt8, 16);
  if (s != MQ_OK) return s;
  if (N < 0 || N > kMaxDim) return fail(MQ_ERR_SHAPE, "N=%lld out of range", (long long)N);
  if (M * N > kMaxElems || K * N > kMaxElems) return fail(MQ_ERR_SHAPE, "problem too large");
  MQ_TRY(need(xq, M * K, "xq"));
  MQ_TRY(need(wq, N * K, "wq"));
  MQ_TRY(need(out, M * N, "the output"));
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(out, 16))
    return fail(MQ_ERR_ALIGN, "xq, wq and the output must be 16-byte aligned");
  (void)out_elem;
  return MQ_OK;
}

}  // namespace

extern "C" {

int mq_abi_version(void) { return MQ_ABI_VERSION; }

const char* mq_status_string(mq_status s) {
  // A C caller may pass any int (a C enum is an int); in C++ a value outside
  // the enumerators' range must not be read as mq_status, so the argument's
  // bytes are read as an int first.
  int v;
  static_assert(sizeof(v) == sizeof(s), "mq_status is passed as an int");
  std::memcpy(&v, &s, sizeof(v));
  switch (v) {
    case MQ_OK: return "MQ_OK";
    case MQ_ERR_NULL: return "MQ_ERR_NULL";
    case MQ_ERR_SHAPE: return "MQ_ERR_SHAPE";
    case MQ_ERR_ALIGN: return "MQ_ERR_ALIGN";
    case MQ_ERR_UNSUPPORTED: return "MQ_ERR_UNSUPPORTED";
    case MQ_ERR_WORKSPACE: return "MQ_ERR_WORKSPACE";
    case MQ_ERR_ALIAS: return "MQ_ERR_ALIAS";
    case MQ_ERR_HIP: return "MQ_ERR_HIP";
  }
  return "MQ_ERR_UNKNOWN";
}

const char* mq_last_error(void) { return g_last_error; }

static mq_status quant_impl(const uint16_t* x, int8_t* xq, float* s_tok, int64_t M, int64_t K, bool bf16,
                            void* stream) {
  mq_status s = check_mk(M, K, 16, kMaxK, 16);
  if (s != MQ_OK) return s;
  MQ_TRY(need(x, M * K, "x"));
  MQ_TRY(need(xq, M * K, "xq"));
  MQ_TRY(need(s_tok, M, "s_tok"));
  if (!aligned(x, 16) || !aligned(xq, 16)) return fail(MQ_ERR_ALIGN, "x and xq must be 16-byte aligned");
  if (!aligned(s_tok, 4)) return fail(MQ_ERR_ALIGN, "s_tok must be 4-byte aligned");
  const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"}};
  const Range out[] = {{xq, static_cast<size_t>(M * K), "xq"}, {s_tok, static_cast<size_t>(M) * 4, "s_tok"}};
  s = check_alias(in, out);
  if (s != MQ_OK) return s;
  if (M == 0) return ok();
  return hip_status(mq::launch_quant_per_token_int8(x, xq, s_tok, M, K, bf16, as_stream(stream)),
                    "quant_per_token_int8 launch");
}

mq_status mq_quant_per_token_int8(const uint16_t* x, int8_t* xq, float* s_tok, int64_t M, int64_t K, void* stream) {
  return quant_impl(x, xq, s_tok, M, K, false, stream);
}

mq_status mq_quant_per_token_int8_bf16(const uint16_t* x, int8_t* xq, float* s_tok, int64_t M, int64_t K,
                                       void* stream) {
  return quant_impl(x, xq, s_tok, M, K, true, stream);
}

static mq_status scaled_mm_impl(const int8_t* xq, const float* s_tok, const int8_t* wq, const float* s_ch, uint16_t* y,
                                int64_t M, int64_t N, int64_t K, bool bf16, void* stream) {
  mq_status s = check_w8a8(xq, wq, y, 2, M, N, K);
  if (s != MQ_OK) return s;
  MQ_TRY(need(s_tok, M, "s_tok"));
  MQ_TRY(need(s_ch, N, "s_ch"));
  if (!aligned(s_tok, 4) || !aligned(s_ch, 4)) return fail(MQ_ERR_ALIGN, "s_tok and s_ch must be 4-byte aligned");
  const Range in[] = {{xq, static_cast<size_t>(M * K), "xq"},
                      {s_tok, static_cast<size_t>(M) * 4, "s_tok"},
                      {wq, static_cast<size_t>(N * K), "wq"},
                      {s_ch, static_cast<size_t>(N) * 4, "s_ch"}};
  const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}};
  s = check_alias(in, out);
  if (s != MQ_OK) return s;
  if (M == 0 || N == 0) return ok();
  return hip_status(mq::launch_w8a8_gemm(xq, s_tok, wq, s_ch, y, nullptr, M, N, K, bf16, as_stream(stream)),
                    "w8a8_scaled_mm launch");
}

mq_status mq_w8a8_scaled_mm(const int8_t* xq, const float* s_tok, const int8_t* wq, const float* s_ch, uint16_t* y,
                            int64_t M, int64_t N, int64_t K, void* stream) {
  return scaled_mm_impl(xq, s_tok, wq, s_ch, y, M, N, K, false, stream);
}

mq_status mq_w8a8_scaled_mm_bf16(const int8_t* xq, const float* s_tok, const int8_t* wq, const float* s_ch,
                                 uint16_t* y, int64_t M, int64_t N, int64_t K, void* stream) {
  return scaled_mm_impl(xq, s_tok, wq, s_ch, y, M, N, K, true, stream);
}

mq_status mq_w8a8_mm_i32(const int8_t* xq, const int8_t* wq, int32_t* acc,
                         int64_t M, int64_t N, int64_t K, void* stream) {
  mq_status s = check_w8a8(xq, wq, acc, 4, M, N, K);
  if (s != MQ_OK) return s;
  const Range in[] = {{xq, static_cast<size_t>(M * K), "xq"}, {wq, static_cast<size_t>(N * K), "wq"}};
  const Range out[] = {{acc, static_cast<size_t>(M * N) * 4, "acc"}};
  s = check_alias(in, out);
  if (s != MQ_OK) return s;
  if (M == 0 || N == 0) return ok();
  return hip_status(mq::launch_w8a8_gemm(xq, nullptr, wq, nullptr, nullptr, acc, M, N, K, false, as_stream(stream)),
                    "w8a8_mm_i32 launch");
}

size_t mq_w4a16_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t group) {
  if (!w4a16_group_ok(group) || M < 1 || M > kMaxDim || N < 8 || N % 8 || N > kMaxN4 ||
      K < 128 || K > kMaxK || K % 128 || M * N > kMaxElems)
    return 0;
  return mq::w4a16_gemm_workspace(M, N, K);
}

static mq_status w4a16_gemm_impl(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                                   const int32_t* qzeros, uint16_t* y, int64_t M, int64_t N, int64_t K,
                                   int64_t group, void* workspace, size_t workspace_bytes, bool bf16, void* stream) {
  mq_status s = check_w4a16(x, qweight, scales, qzeros, y, M, N, K, group);
  if (s != MQ_OK) return s;
  if (M == 0) return ok();
  // A workspace is optional: given (large enough for the split plan), K may
  // be split for small tile grids; NULL never splits.
  void* ws = nullptr;
  if (workspace != nullptr) {
    const size_t need = mq::w4a16_gemm_workspace(M, N, K);
    if (need > 0) {
      if (workspace_bytes < need)
        return fail(MQ_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
      if (!aligned(workspace, 16)) return fail(MQ_ERR_ALIGN, "workspace must be 16-byte aligned");
      const size_t G = group_rows(K, group);
      const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"},
                          {qweight, static_cast<size_t>(K * (N / 8)) * 4, "qweight"},
                          {scales, G * static_cast<size_t>(N) * 2, "scales"},
                          {qzeros, G * static_cast<size_t>(N / 8) * 4, "qzeros"}};
      const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}, {workspace, need, "workspace"}};
      s = check_alias(in, out);
      if (s != MQ_OK) return s;
      ws = workspace;
    }
  }
  return hip_status(mq::launch_w4a16_gemm(x, qweight, scales, qzeros, y, M, N, K, kernel_group(group), group == -1,
                                          ws, bf16, as_stream(stream)),
                    "w4a16_gemm launch");
}

size_t mq_w4a16_gemv_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t group) {
  if (!w4a16_group_ok(group) || M < 1 || M > mq::kGemvMaxM || N < 8 || N % 8 ||
      N > kMaxN4 || K < 128 || K > kMaxK || K % 128)
    return 0;
  return mq::plan_w4a16_gemv(M, N, K, kernel_group(group)).workspace_bytes;
}

static mq_status w4a16_gemv_impl(const uint16_t* x, const int32_t* qweight, const uint16_t* scales,
                                   const int32_t* qzeros, uint16_t* y, int64_t M, int64_t N, int64_t K,
                                   int64_t group, void* workspace, size_t workspace_bytes, bool bf16, void* stream) {
  mq_status s = check_w4a16(x, qweight, scales, qzeros, y, M, N, K, group);
  if (s != MQ_OK) return s;
  if (M > mq::kGemvMaxM)
    return fail(MQ_ERR_UNSUPPORTED, "GEMV needs M <= %lld (got %lld); use mq_w4a16_gemm",
                (long long)mq::kGemvMaxM, (long long)M);
  if (M == 0) return ok();
  mq::GemvPlan plan = mq::plan_w4a16_gemv(M, N, K, kernel_group(group));
  plan.per_channel = group == -1;
  if (plan.workspace_bytes > 0) {
    if (!workspace || workspace_bytes < plan.workspace_bytes)
      return fail(MQ_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", plan.workspace_bytes,
                  workspace ? workspace_bytes : static_cast<size_t>(0));
    if (!aligned(workspace, 16)) return fail(MQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    const size_t G = group_rows(K, group);
    const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"},
                        {qweight, static_cast<size_t>(K * (N / 8)) * 4, "qweight"},
                        {scales, G * static_cast<size_t>(N) * 2, "scales"},
                        {qzeros, G * static_cast<size_t>(N / 8) * 4, "qzeros"}};
    const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}, {workspace, plan.workspace_bytes, "workspace"}};
    s = check_alias(in, out);
    if (s != MQ_OK) return s;
  }
  return hip_status(mq::launch_w4a16_gemv(x, qweight, scales, qzeros, y, M, N, K, plan,
                                          plan.workspace_bytes ? workspace : nullptr, bf16, as_stream(stream)),
                    "w4a16_gemv launch");
}

static mq_status kv_quant_impl(const uint16_t* x, uint8_t* codes, float* params, int64_t rows, int64_t head_dim,
                               int32_t bits, bool bf16, void* stream) {
  if (bits != 8 && bits != 4) return fail(MQ_ERR_UNSUPPORTED, "bits=%d (8 and 4 are provided)", (int)bits);
  if (head_dim < 8 || head_dim > 512 || (head_dim & (head_dim - 1)))
    return fail(MQ_ERR_SHAPE, "head_dim=%lld must be a power of two in [8, 512]", (long long)head_dim);
  if (rows < 0 || rows > kMaxDim) return fail(MQ_ERR_SHAPE, "rows=%lld out of range", (long long)rows);
  // one lane per 8 values: the launch holds rows * head_dim / 8 < 2^32 work-items
  if (rows * head_dim >= (int64_t{1} << 35))
    return fail(MQ_ERR_SHAPE, "rows * head_dim = %lld must be below 2^35", (long long)(rows * head_dim));
  MQ_TRY(need(x, rows * head_dim, "x"));
  MQ_TRY(need(codes, rows * head_dim, "codes"));
  MQ_TRY(need(params, rows, "params"));
  if (!aligned(x, 16)) return fail(MQ_ERR_ALIGN, "x must be 16-byte aligned");
  if (!aligned(codes, bits == 8 ? 8 : 4)) return fail(MQ_ERR_ALIGN, "codes must be %d-byte aligned", bits == 8 ? 8 : 4);
  if (!aligned(params, 8)) return fail(MQ_ERR_ALIGN, "params must be 8-byte aligned");
  const Range in[] = {{x, static_cast<size_t>(rows * head_dim) * 2, "x"}};
  const Range out[] = {{codes, static_cast<size_t>(rows * head_dim) * bits / 8, "codes"},
                       {params, static_cast<size_t>(rows) * 8, "params"}};
  MQ_TRY(check_alias(in, out));
  if (rows == 0) return ok();
  return hip_status(mq::launch_kv_quant(x, codes, params, rows, head_dim, bits, bf16, as_stream(stream)),
                    "kv_quant launch");
}

mq_status mq_kv_quant(const uint16_t* x, uint8_t* codes, float* params, int64_t rows, int64_t head_dim,
                      int32_t bits, void* stream) {
  return kv_quant_impl(x, codes, params, rows, head_dim, bits, false, stream);
}

mq_status mq_kv_quant_bf16(const uint16_t* x, uint8_t* codes, float* params, int64_t rows, int64_t head_dim,
                           int32_t bits, void* stream) {
  return kv_quant_impl(x, codes, params, rows, head_dim, bits, true, stream);
}

namespace {

// A field order: NULL means the library's own (field j = element j);
// otherwise a permutation of 0..7.
mq_status field_order(const uint8_t* order, uint8_t (&out)[8]) {
  for (int j = 0; j < 8; ++j) out[j] = static_cast<uint8_t>(j);
  if (order == nullptr) return MQ_OK;
  unsigned seen = 0;
  for (int j = 0; j < 8; ++j) {
    if (order[j] > 7 || (seen >> order[j]) & 1u)
      return fail(MQ_ERR_UNSUPPORTED, "field_order must be a permutation of 0..7");
    seen |= 1u << order[j];
    out[j] = order[j];
  }
  return MQ_OK;
}

}  // namespace

mq_status mq_int4_reorder(const int32_t* src, int32_t* dst, int64_t words, const uint8_t* order, void* stream) {
  uint8_t ord[8];
  MQ_TRY(field_order(order, ord));
  if (words < 0 || words >= (int64_t{1} << 34))
    return fail(MQ_ERR_SHAPE, "words=%lld out of range", (long long)words);
  MQ_TRY(need(src, words, "src"));
  MQ_TRY(need(dst, words, "dst"));
  if (!aligned(src, 16) || !aligned(dst, 16)) return fail(MQ_ERR_ALIGN, "src and dst must be 16-byte aligned");
  const Range in[] = {{src, static_cast<size_t>(words) * 4, "src"}};
  const Range out[] = {{dst, static_cast<size_t>(words) * 4, "dst"}};
  MQ_TRY(check_alias(in, out));
  if (words == 0) return ok();
  return hip_status(mq::launch_int4_reorder(src, dst, words, ord, as_stream(stream)), "int4_reorder launch");
}

mq_status mq_int4_transpose(const int32_t* src, int32_t* dst, int64_t A, int64_t B, const uint8_t* order,
                            void* stream) {
  uint8_t ord[8];
  MQ_TRY(field_order(order, ord));
  if (A < 0 || B < 0 || A % 8 || B % 8)
    return fail(MQ_ERR_SHAPE, "A=%lld and B=%lld must be non-negative multiples of 8", (long long)A, (long long)B);
  if (A > mq::kInt4TransposeMaxA || B > kMaxDim || A * B > kMaxElems)
    return fail(MQ_ERR_SHAPE, "A=%lld, B=%lld too large", (long long)A, (long long)B);
  MQ_TRY(need(src, A * B, "src"));
  MQ_TRY(need(dst, A * B, "dst"));
  if (!aligned(src, 4) || !aligned(dst, 4)) return fail(MQ_ERR_ALIGN, "src and dst must be 4-byte aligned");
  const Range in[] = {{src, static_cast<size_t>(A * B) / 2, "src"}};
  const Range out[] = {{dst, static_cast<size_t>(A * B) / 2, "dst"}};
  MQ_TRY(check_alias(in, out));
  if (A == 0 || B == 0) return ok();
  return hip_status(mq::launch_int4_transpose(src, dst, A, B, ord, as_stream(stream)), "int4_transpose launch");
}

mq_status mq_u16_transpose(const uint16_t* src, uint16_t* dst, int64_t A, int64_t B, void* stream) {
  if (A < 0 || B < 0 || A > mq::kU16TransposeMaxA || B > mq::kU16TransposeMaxB || A * B > kMaxElems)
    return fail(MQ_ERR_SHAPE, "A=%lld, B=%lld out of range", (long long)A, (long long)B);
  MQ_TRY(need(src, A * B, "src"));
  MQ_TRY(need(dst, A * B, "dst"));
  if (!aligned(src, 2) || !aligned(dst, 2)) return fail(MQ_ERR_ALIGN, "src and dst must be 2-byte aligned");
  const Range in[] = {{src, static_cast<size_t>(A * B) * 2, "src"}};
  const Range out[] = {{dst, static_cast<size_t>(A * B) * 2, "dst"}};
  MQ_TRY(check_alias(in, out));
  if (A == 0 || B == 0) return ok();
  return hip_status(mq::launch_u16_transpose(src, dst, A, B, as_stream(stream)), "u16_transpose launch");
}

// The workspace does not depend on N: it is sized for the two-kernel path,
// which every M can take (the one-kernel path for 1-4 tokens leaves it
// unused).
size_t mq_w8a8_linear_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || M > kMaxDim || K < 16 || K > kMaxKInt8 || K % 16 || M * K > kMaxElems || M == 0) return 0;
  return (static_cast<size_t>(M * K) + 255) / 256 * 256 + static_cast<size_t>(M) * 4;
}

static_assert(mq::kNoallocScratchBytes == MQ_NOALLOC_SCRATCH_BYTES, "scratch size in mq.h");

// noalloc: the workspace is the library's scratch array, looked up after
// every argument check passed (the only HIP call before the launches).
static mq_status linear_impl(const uint16_t* x, const int8_t* wq, const float* s_ch, uint16_t* y, int64_t M,
                             int64_t N, int64_t K, void* workspace, size_t workspace_bytes, bool bf16, void* stream,
                             bool noalloc = false) {
  mq_status s = check_mk(M, K, 16, kMaxKInt8, 16);
  if (s != MQ_OK) return s;
  if (N < 0 || N > kMaxDim) return fail(MQ_ERR_SHAPE, "N=%lld out of range", (long long)N);
  if (M * N > kMaxElems || K * N > kMaxElems) return fail(MQ_ERR_SHAPE, "problem too large");
  MQ_TRY(need(x, M * K, "x"));
  MQ_TRY(need(wq, N * K, "wq"));
  MQ_TRY(need(s_ch, N, "s_ch"));
  MQ_TRY(need(y, M * N, "y"));
  if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(y, 16))
    return fail(MQ_ERR_ALIGN, "x, wq and y must be 16-byte aligned");
  if (!aligned(s_ch, 4)) return fail(MQ_ERR_ALIGN, "s_ch must be 4-byte aligned");
  const bool fused = mq::w8a8_use_fused(M, N, K);
  const size_t ws = fused ? 0 : mq_w8a8_linear_workspace_bytes(M, K);
  if (noalloc) {
    if (ws > MQ_NOALLOC_SCRATCH_BYTES)
      return fail(MQ_ERR_WORKSPACE, "M*K=%lld needs %zu bytes of scratch; the allocation-free entry holds %zu",
                  (long long)(M * K), ws, static_cast<size_t>(MQ_NOALLOC_SCRATCH_BYTES));
  } else if (ws > 0) {
    if (!workspace || workspace_bytes < ws)
      return fail(MQ_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", ws,
                  workspace ? workspace_bytes : static_cast<size_t>(0));
    if (!aligned(workspace, 16)) return fail(MQ_ERR_ALIGN, "workspace must be 16-byte aligned");
  }
  const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"},
                      {wq, static_cast<size_t>(N * K), "wq"},
                      {s_ch, static_cast<size_t>(N) * 4, "s_ch"}};
  // (the library's scratch cannot overlap a caller's buffer)
  const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"},
                       {ws && !noalloc ? workspace : nullptr, noalloc ? 0 : ws, "workspace"}};
  s = check_alias(in, out);
  if (s != MQ_OK) return s;
  if (M == 0 || N == 0) return ok();
  if (noalloc && ws > 0) {
    MQ_TRY(hip_status(mq::noalloc_scratch(&workspace), "w8a8_linear_noalloc scratch lookup"));
    workspace_bytes = MQ_NOALLOC_SCRATCH_BYTES;
  }
  if (fused)
    return hip_status(mq::launch_w8a8_gemv_fused(x, wq, s_ch, y, M, N, K, bf16, as_stream(stream)),
                      "w8a8_linear launch");
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* s_tok = reinterpret_cast<float*>(static_cast<char*>(workspace) + (static_cast<size_t>(M * K) + 255) / 256 * 256);
  s = hip_status(mq::launch_quant_per_token_int8(x, xq, s_tok, M, K, bf16, as_stream(stream)),
                 "w8a8_linear quant launch");
  if (s != MQ_OK) return s;
  return hip_status(mq::launch_w8a8_gemm(xq, s_tok, wq, s_ch, y, nullptr, M, N, K, bf16, as_stream(stream)),
                    "w8a8_linear gemm launch");
}

mq_status mq_w8a8_linear(const uint16_t* x, const int8_t* wq, const float* s_ch, uint16_t* y, int64_t M, int64_t N,
                         int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return linear_impl(x, wq, s_ch, y, M, N, K, workspace, workspace_bytes, false, stream);
}

mq_status mq_w8a8_linear_bf16(const uint16_t* x, const int8_t* wq, const float* s_ch, uint16_t* y, int64_t M,
                              int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return linear_impl(x, wq, s_ch, y, M, N, K, workspace, workspace_bytes, true, stream);
}

mq_status mq_w8a8_linear_noalloc(const uint16_t* x, const int8_t* wq, const float* s_ch, uint16_t* y, int64_t M,
                                 int64_t N, int64_t K, void* stream) {
  return linear_impl(x, wq, s_ch, y, M, N, K, nullptr, 0, false, stream, true);
}

mq_status mq_w4a16_block_weights(const int32_t* qweight, int32_t* qweight_blocked, int64_t N, int64_t K,
                                 void* stream) {
  if (N < 0 || N > kMaxN4 || N % 32)
    return fail(MQ_ERR_SHAPE, "N=%lld must be a multiple of 32 in [0, 2^27]", (long long)N);
  if (K < 0 || K > kMaxK || K % 128)
    return fail(MQ_ERR_SHAPE, "K=%lld must be a multiple of 128 in [0, 2^20]", (long long)K);
  if (K * N > kMaxElems) return fail(MQ_ERR_SHAPE, "problem too large");
  MQ_TRY(need(qweight, K * N, "qweight"));
  MQ_TRY(need(qweight_blocked, K * N, "qweight_blocked"));
  if (!aligned(qweight, 4)) return fail(MQ_ERR_ALIGN, "qweight must be 4-byte aligned");
  if (!aligned(qweight_blocked, 16)) return fail(MQ_ERR_ALIGN, "qweight_blocked must be 16-byte aligned");
  const size_t bytes = static_cast<size_t>(K * (N / 8)) * 4;
  const Range in[] = {{qweight, bytes, "qweight"}};
  const Range out[] = {{qweight_blocked, bytes, "qweight_blocked"}};
  MQ_TRY(check_alias(in, out));
  if (K == 0 || N == 0) return ok();
  return hip_status(mq::launch_w4a16_block_weights(qweight, qweight_blocked, N, K, as_stream(stream)),
                    "w4a16_block_weights launch");
}

// The decode-layout kernels address the scale and zero-point tables with
// 32-bit buffer offsets.
constexpr size_t kMaxScaleBytes = (size_t{1} << 31) - 1;
static bool blocked_scales_fit(int64_t N, int64_t K, int64_t group) {
  return group_rows(K, group) * static_cast<size_t>(N) * 2 <= kMaxScaleBytes;
}

size_t mq_w4a16_gemv_blocked_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t group) {
  if (!w4a16_group_ok(group) || M < 1 || M > mq::kGemvMaxM || N < 32 || N % 32 ||
      N > kMaxN4 || K < 128 || K > kMaxK || K % 128 || !blocked_scales_fit(N, K, group))
    return 0;
  return mq::w4a16_gemv_blocked_workspace(M, N, K, kernel_group(group));
}

static mq_status w4a16_gemv_blocked_impl(const uint16_t* x, const int32_t* qweight_blocked,
                                         const uint16_t* scales, const int32_t* qzeros, uint16_t* y, int64_t M,
                                         int64_t N, int64_t K, int64_t group, void* workspace,
                                         size_t workspace_bytes, bool bf16, void* stream) {
  mq_status s = check_w4a16(x, qweight_blocked, scales, qzeros, y, M, N, K, group);
  if (s != MQ_OK) return s;
  if (N % 32) return fail(MQ_ERR_SHAPE, "the blocked layout needs N %% 32 == 0 (got N=%lld)", (long long)N);
  if (!blocked_scales_fit(N, K, group))
    return fail(MQ_ERR_SHAPE, "scales of %zu bytes: the decode-layout GEMV takes at most 2^31 - 1",
                group_rows(K, group) * static_cast<size_t>(N) * 2);
  if (!aligned(qweight_blocked, 16)) return fail(MQ_ERR_ALIGN, "qweight_blocked must be 16-byte aligned");
  if (M > mq::kGemvMaxM)
    return fail(MQ_ERR_UNSUPPORTED, "GEMV needs M <= %lld (got %lld); use mq_w4a16_gemm",
                (long long)mq::kGemvMaxM, (long long)M);
  if (M == 0) return ok();
  const size_t need_ws = mq::w4a16_gemv_blocked_workspace(M, N, K, kernel_group(group));
  if (need_ws > 0) {
    if (!workspace || workspace_bytes < need_ws)
      return fail(MQ_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need_ws,
                  workspace ? workspace_bytes : static_cast<size_t>(0));
    if (!aligned(workspace, 16)) return fail(MQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    const size_t G = group_rows(K, group);
    const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"},
                        {qweight_blocked, static_cast<size_t>(K * (N / 8)) * 4, "qweight_blocked"},
                        {scales, G * static_cast<size_t>(N) * 2, "scales"},
                        {qzeros, G * static_cast<size_t>(N / 8) * 4, "qzeros"}};
    const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}, {workspace, need_ws, "workspace"}};
    s = check_alias(in, out);
    if (s != MQ_OK) return s;
  }
  mq::GemvPlan plan = mq::plan_w4a16_gemv_blocked(M, N, K, kernel_group(group));
  plan.per_channel = group == -1;
  return hip_status(mq::launch_w4a16_gemv_blocked(x, qweight_blocked, scales, qzeros, y, M, N, K, plan,
                                                  need_ws ? workspace : nullptr, bf16, as_stream(stream)),
                    "w4a16_gemv_blocked launch");
}

#define MQ_W4A16_ENTRY(NAME, IMPL, BF, WNAME)                                                                  \
  mq_status NAME(const uint16_t* x, const int32_t* WNAME, const uint16_t* scales, const int32_t* qzeros,       \
                 uint16_t* y, int64_t M, int64_t N, int64_t K, int64_t group, void* workspace,                  \
                 size_t workspace_bytes, void* stream) {                                                        \
    return IMPL(x, WNAME, scales, qzeros, y, M, N, K, group, workspace, workspace_bytes, BF, stream);         \
  }
MQ_W4A16_ENTRY(mq_w4a16_gemm, w4a16_gemm_impl, false, qweight)
MQ_W4A16_ENTRY(mq_w4a16_gemm_bf16, w4a16_gemm_impl, true, qweight)
MQ_W4A16_ENTRY(mq_w4a16_gemv, w4a16_gemv_impl, false, qweight)
MQ_W4A16_ENTRY(mq_w4a16_gemv_bf16, w4a16_gemv_impl, true, qweight)
MQ_W4A16_ENTRY(mq_w4a16_gemv_blocked, w4a16_gemv_blocked_impl, false, qweight_blocked)
MQ_W4A16_ENTRY(mq_w4a16_gemv_blocked_bf16, w4a16_gemv_blocked_impl, true, qweight_blocked)
#undef MQ_W4A16_ENTRY

// ---- RMS norm with 8-bit output, e4m3 codes and product -------------------

static size_t blocks_of(int64_t n) { return static_cast<size_t>((n + 127) / 128); }

static mq_status rmsnorm_impl(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps,
                              uint16_t* h, void* codes, float* scales, int64_t M, int64_t K, bool fp8, bool bf16,
                              void* stream) {
  MQ_TRY(check_mk(M, K, 16, mq::kRmsnormMaxK, 16));
  if (M >= (int64_t{1} << 22)) return fail(MQ_ERR_SHAPE, "M=%lld must be below 2^22", (long long)M);
  if (!(eps >= 0.0 && eps <= 1.0)) return fail(MQ_ERR_UNSUPPORTED, "eps=%g must lie in [0, 1]", eps);
  MQ_TRY(need(x, M * K, "x"));
  MQ_TRY(need(weight, K, "weight"));
  MQ_TRY(need(codes, M * K, "xq"));
  MQ_TRY(need(scales, M, "the scales"));
  if (M > 0 && (residual == nullptr) != (h == nullptr))
    return fail(MQ_ERR_NULL, "residual and h are given together or not at all");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16))
    return fail(MQ_ERR_ALIGN, "x, residual, weight and h must be 16-byte aligned");
  if (!aligned(codes, 16)) return fail(MQ_ERR_ALIGN, "xq must be 16-byte aligned");
  if (!aligned(scales, 4)) return fail(MQ_ERR_ALIGN, "the scales must be 4-byte aligned");
  const size_t n = static_cast<size_t>(M * K), ns = static_cast<size_t>(M) * (fp8 ? blocks_of(K) : 1) * 4;
  // h may be the residual itself (each value is read before it is replaced,
  // by the same lane); any other overlap is an error.
  const bool in_place = h == residual;
  const Range in[] = {{x, n * 2, "x"},
                      {in_place ? nullptr : residual, in_place || residual == nullptr ? 0 : n * 2, "residual"},
                      {weight, static_cast<size_t>(K) * 2, "weight"}};
  const Range out[] = {{h, h ? n * 2 : 0, "h"}, {codes, n, "xq"}, {scales, ns, "the scales"}};
  MQ_TRY(check_alias(in, out));
  if (M == 0) return ok();
  return hip_status(mq::launch_rmsnorm_quant(x, residual, weight, eps, h, static_cast<uint8_t*>(codes), scales, M, K, fp8,
                                             bf16, as_stream(stream)),
                    "rmsnorm launch");
}

mq_status mq_rmsnorm_int8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps, uint16_t* h,
                          int8_t* xq, float* s_tok, int64_t M, int64_t K, void* stream) {
  return rmsnorm_impl(x, residual, weight, eps, h, xq, s_tok, M, K, false, false, stream);
}

mq_status mq_rmsnorm_int8_bf16(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps,
                               uint16_t* h, int8_t* xq, float* s_tok, int64_t M, int64_t K, void* stream) {
  return rmsnorm_impl(x, residual, weight, eps, h, xq, s_tok, M, K, false, true, stream);
}

mq_status mq_rmsnorm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps, uint16_t* h,
                         uint8_t* xq, float* s_x, int64_t M, int64_t K, void* stream) {
  return rmsnorm_impl(x, residual, weight, eps, h, xq, s_x, M, K, true, false, stream);
}

mq_status mq_rmsnorm_fp8_bf16(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, double eps,
                              uint16_t* h, uint8_t* xq, float* s_x, int64_t M, int64_t K, void* stream) {
  return rmsnorm_impl(x, residual, weight, eps, h, xq, s_x, M, K, true, true, stream);
}

// one 16-lane group per block of 128: the launch holds 16 M ceil(K / 128) < 2^32 work-items
static mq_status check_fp8_rows(int64_t M, int64_t K) {
  MQ_TRY(check_mk(M, K, 16, kMaxK, 16));
  if (M * static_cast<int64_t>(blocks_of(K)) >= (int64_t{1} << 27))
    return fail(MQ_ERR_SHAPE, "M * ceil(K / 128) = %lld must be below 2^27", (long long)(M * (int64_t)blocks_of(K)));
  return MQ_OK;
}

static mq_status quant_fp8_impl(const uint16_t* x, uint8_t* xq, float* s_x, int64_t M, int64_t K, bool bf16,
                                void* stream) {
  MQ_TRY(check_fp8_rows(M, K));
  MQ_TRY(need(x, M * K, "x"));
  MQ_TRY(need(xq, M * K, "xq"));
  MQ_TRY(need(s_x, M, "s_x"));
  if (!aligned(x, 16) || !aligned(xq, 16)) return fail(MQ_ERR_ALIGN, "x and xq must be 16-byte aligned");
  if (!aligned(s_x, 4)) return fail(MQ_ERR_ALIGN, "s_x must be 4-byte aligned");
  const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"}};
  const Range out[] = {{xq, static_cast<size_t>(M * K), "xq"}, {s_x, static_cast<size_t>(M) * blocks_of(K) * 4, "s_x"}};
  MQ_TRY(check_alias(in, out));
  if (M == 0) return ok();
  return hip_status(mq::launch_quant_fp8_blocks(x, xq, s_x, M, K, bf16, as_stream(stream)), "quant_fp8_blocks launch");
}

mq_status mq_quant_fp8_blocks(const uint16_t* x, uint8_t* xq, float* s_x, int64_t M, int64_t K, void* stream) {
  return quant_fp8_impl(x, xq, s_x, M, K, false, stream);
}

mq_status mq_quant_fp8_blocks_bf16(const uint16_t* x, uint8_t* xq, float* s_x, int64_t M, int64_t K, void* stream) {
  return quant_fp8_impl(x, xq, s_x, M, K, true, stream);
}

constexpr int64_t kMaxFp8Dim = int64_t{1} << 26;    // M, N of the e4m3 product (launch size)
constexpr int64_t kMaxFp8Out = int64_t{1} << 36;    // M * N of it

static bool fp8_mm_sizes(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && M <= kMaxFp8Dim && N >= 0 && N <= kMaxFp8Dim && K >= 16 && K <= kMaxK && K % 16 == 0 &&
         M * N <= kMaxFp8Out && M * K <= kMaxElems && K * N <= kMaxElems;
}

static mq_status check_fp8_mm(int64_t M, int64_t N, int64_t K) {
  MQ_TRY(check_mk(M, K, 16, kMaxK, 16));
  if (M > kMaxFp8Dim) return fail(MQ_ERR_SHAPE, "M=%lld out of range", (long long)M);
  if (N < 0 || N > kMaxFp8Dim) return fail(MQ_ERR_SHAPE, "N=%lld out of range", (long long)N);
  if (!fp8_mm_sizes(M, N, K)) return fail(MQ_ERR_SHAPE, "problem too large");
  return MQ_OK;
}

static mq_status check_workspace(const void* workspace, size_t given, size_t needed) {
  if (needed == 0) return MQ_OK;
  if (!workspace || given < needed)
    return fail(MQ_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", needed, workspace ? given : static_cast<size_t>(0));
  if (!aligned(workspace, 16)) return fail(MQ_ERR_ALIGN, "workspace must be 16-byte aligned");
  return MQ_OK;
}

static mq_status fp8_mm_impl(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, bool bf16,
                             void* stream) {
  MQ_TRY(check_fp8_mm(M, N, K));
  MQ_TRY(need(xq, M * K, "xq"));
  MQ_TRY(need(s_x, M, "s_x"));
  MQ_TRY(need(wq, N * K, "wq"));
  MQ_TRY(need(s_w, N, "s_w"));
  MQ_TRY(need(y, M * N, "y"));
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(y, 16))
    return fail(MQ_ERR_ALIGN, "xq, wq and y must be 16-byte aligned");
  if (!aligned(s_x, 4) || !aligned(s_w, 4)) return fail(MQ_ERR_ALIGN, "s_x and s_w must be 4-byte aligned");
  const bool empty = M == 0 || N == 0;
  const mq::Fp8Plan plan = empty ? mq::Fp8Plan{} : mq::plan_fp8_block_mm(M, N, K);
  MQ_TRY(check_workspace(workspace, workspace_bytes, plan.workspace_bytes));
  const Range in[] = {{xq, static_cast<size_t>(M * K), "xq"},
                      {s_x, static_cast<size_t>(M) * blocks_of(K) * 4, "s_x"},
                      {wq, static_cast<size_t>(N * K), "wq"},
                      {s_w, blocks_of(N) * blocks_of(K) * 4, "s_w"}};
  const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}, {workspace, plan.workspace_bytes, "workspace"}};
  MQ_TRY(check_alias(in, out));
  if (empty) return ok();
  return hip_status(mq::launch_fp8_block_mm(xq, s_x, wq, s_w, y, M, N, K, plan, workspace, bf16, as_stream(stream)),
                    "fp8_block_mm launch");
}

size_t mq_fp8_block_mm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!fp8_mm_sizes(M, N, K) || M == 0 || N == 0) return 0;
  return mq::plan_fp8_block_mm(M, N, K).workspace_bytes;
}

mq_status mq_fp8_block_mm(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                          int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return fp8_mm_impl(xq, s_x, wq, s_w, y, M, N, K, workspace, workspace_bytes, false, stream);
}

mq_status mq_fp8_block_mm_bf16(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y,
                               int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return fp8_mm_impl(xq, s_x, wq, s_w, y, M, N, K, workspace, workspace_bytes, true, stream);
}

// fp8_linear's workspace: the codes, the scales, the product's own part. None
// where one kernel does it all.
struct Fp8LinearPlan {
  mq::Fp8Plan mm;
  bool fused;
  size_t scales_at, mm_at, bytes;
};
static Fp8LinearPlan fp8_linear_plan(int64_t M, int64_t N, int64_t K) {
  Fp8LinearPlan p = {};
  if (M == 0 || N == 0) return p;
  p.mm = mq::plan_fp8_block_mm(M, N, K);
  p.fused = mq::fp8_use_fused(M, K);
  if (p.fused) return p;
  p.scales_at = (static_cast<size_t>(M * K) + 255) / 256 * 256;
  p.mm_at = (p.scales_at + static_cast<size_t>(M) * blocks_of(K) * 4 + 255) / 256 * 256;
  p.bytes = p.mm_at + p.mm.workspace_bytes;
  return p;
}

size_t mq_fp8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return fp8_mm_sizes(M, N, K) ? fp8_linear_plan(M, N, K).bytes : 0;
}

static mq_status fp8_linear_impl(const uint16_t* x, const uint8_t* wq, const float* s_w, uint16_t* y, int64_t M,
                                 int64_t N, int64_t K, void* workspace, size_t workspace_bytes, bool bf16,
                                 void* stream) {
  MQ_TRY(check_fp8_mm(M, N, K));
  MQ_TRY(check_fp8_rows(M, K));
  MQ_TRY(need(x, M * K, "x"));
  MQ_TRY(need(wq, N * K, "wq"));
  MQ_TRY(need(s_w, N, "s_w"));
  MQ_TRY(need(y, M * N, "y"));
  if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(y, 16))
    return fail(MQ_ERR_ALIGN, "x, wq and y must be 16-byte aligned");
  if (!aligned(s_w, 4)) return fail(MQ_ERR_ALIGN, "s_w must be 4-byte aligned");
  const Fp8LinearPlan plan = fp8_linear_plan(M, N, K);
  MQ_TRY(check_workspace(workspace, workspace_bytes, plan.bytes));
  const Range in[] = {{x, static_cast<size_t>(M * K) * 2, "x"},
                      {wq, static_cast<size_t>(N * K), "wq"},
                      {s_w, blocks_of(N) * blocks_of(K) * 4, "s_w"}};
  const Range out[] = {{y, static_cast<size_t>(M * N) * 2, "y"}, {workspace, plan.bytes, "workspace"}};
  MQ_TRY(check_alias(in, out));
  if (M == 0 || N == 0) return ok();
  if (plan.fused)
    return hip_status(mq::launch_fp8_block_gemv(x, nullptr, nullptr, wq, s_w, y, M, N, K, bf16, as_stream(stream)),
                      "fp8_linear launch");
  uint8_t* const xq = static_cast<uint8_t*>(workspace);
  float* const s_x = reinterpret_cast<float*>(xq + plan.scales_at);
  MQ_TRY(hip_status(mq::launch_quant_fp8_blocks(x, xq, s_x, M, K, bf16, as_stream(stream)), "fp8_linear quant launch"));
  return hip_status(mq::launch_fp8_block_mm(xq, s_x, wq, s_w, y, M, N, K, plan.mm, xq + plan.mm_at, bf16,
                                            as_stream(stream)),
                    "fp8_linear mm launch");
}

mq_status mq_fp8_linear(const uint16_t* x, const uint8_t* wq, const float* s_w, uint16_t* y, int64_t M, int64_t N,
                        int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return fp8_linear_impl(x, wq, s_w, y, M, N, K, workspace, workspace_bytes, false, stream);
}

mq_status mq_fp8_linear_bf16(const uint16_t* x, const uint8_t* wq, const float* s_w, uint16_t* y, int64_t M, int64_t N,
                             int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return fp8_linear_impl(x, wq, s_w, y, M, N, K, workspace, workspace_bytes, true, stream);
}

// ---- paged e4m3 KV cache ---------------------------------------------------

// Everything but the rows of q, k and v. T == 0 or B == 0 is an empty call.
static mq_status kv8_cache(const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scales, const float* v_scales,
                           const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int64_t B,
                           int64_t Hkv, int64_t D, int64_t page, int64_t num_pages, int64_t table_width,
                           int64_t max_q_len, mq::Kv8Cache& c) {
  if (D != 64 && D != 128) return fail(MQ_ERR_UNSUPPORTED, "head_dim=%lld (64 and 128 are provided)", (long long)D);
  if (page != 16 && page != 32 && page != 64 && page != 128)
    return fail(MQ_ERR_UNSUPPORTED, "page=%lld (16, 32, 64 and 128 tokens are provided)", (long long)page);
  if (T < 0 || T > (int64_t{1} << 26)) return fail(MQ_ERR_SHAPE, "T=%lld out of range", (long long)T);
  if (B < 0 || B > 65535) return fail(MQ_ERR_SHAPE, "B=%lld must lie in [0, 65535]", (long long)B);
  if (Hkv < 1 || Hkv > 1024) return fail(MQ_ERR_SHAPE, "Hkv=%lld must lie in [1, 1024]", (long long)Hkv);
  if (num_pages < 1 || num_pages > kMaxDim) return fail(MQ_ERR_SHAPE, "num_pages=%lld out of range", (long long)num_pages);
  if (table_width < 1 || table_width > (int64_t{1} << 30) / page)
    return fail(MQ_ERR_SHAPE, "table_width=%lld: a sequence holds at most 2^30 tokens", (long long)table_width);
  if (max_q_len < 1 || max_q_len > kMaxDim) return fail(MQ_ERR_SHAPE, "max_q_len=%lld must be positive", (long long)max_q_len);
  MQ_TRY(need(k_cache, 1, "k_cache"));
  MQ_TRY(need(v_cache, 1, "v_cache"));
  MQ_TRY(need(k_scales, 1, "k_scales"));
  MQ_TRY(need(v_scales, 1, "v_scales"));
  MQ_TRY(need(block_table, B, "block_table"));
  MQ_TRY(need(cu_q, B, "cu_q"));
  MQ_TRY(need(kv_lens, B, "kv_lens"));
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return fail(MQ_ERR_ALIGN, "k_cache and v_cache must be 16-byte aligned");
  if (!aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4))
    return fail(MQ_ERR_ALIGN, "scales, block_table, cu_q and kv_lens must be 4-byte aligned");
  c = {};
  c.k = const_cast<uint8_t*>(k_cache);
  c.v = const_cast<uint8_t*>(v_cache);
  c.k_scales = const_cast<float*>(k_scales);
  c.v_scales = const_cast<float*>(v_scales);
  c.table = block_table;
  c.cu = cu_q;
  c.lens = kv_lens;
  c.batch = static_cast<int>(B);
  c.kv_heads = static_cast<int>(Hkv);
  c.head_dim = static_cast<int>(D);
  c.page = static_cast<int>(page);
  for (c.page_shift = 4; (1 << c.page_shift) < c.page;) ++c.page_shift;
  c.num_pages = static_cast<int>(num_pages);
  c.table_width = static_cast<int>(table_width);
  c.tokens = static_cast<int>(T);
  c.max_q_len = static_cast<int>(max_q_len);
  return MQ_OK;
}

// Rows of `width` 16-bit values, `stride` values apart.
static mq_status kv8_rows(const uint16_t* p, int64_t T, int64_t width, int64_t stride, const char* name, size_t& bytes) {
  MQ_TRY(need(p, T, name));
  if (stride < width || stride % 8 || stride > kMaxDim)
    return fail(MQ_ERR_SHAPE, "%s: a stride of %lld for rows of %lld values (a multiple of 8, no less than the row)", name,
                (long long)stride, (long long)width);
  if (!aligned(p, 16)) return fail(MQ_ERR_ALIGN, "%s must be 16-byte aligned", name);
  bytes = T > 0 ? (static_cast<size_t>(T - 1) * stride + width) * 2 : 0;
  return MQ_OK;
}

static mq_status kv8_append_impl(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                                 uint8_t* k_cache, uint8_t* v_cache, float* k_scales, float* v_scales,
                                 const int32_t* block_table, const int32_t* cu_q, const int32_t* kv_lens, int64_t T,
                                 int64_t B, int64_t Hkv, int64_t D, int64_t page, int64_t num_pages,
                                 int64_t table_width, int64_t max_q_len, bool bf16, void* stream) {
  mq::Kv8Cache c;
  MQ_TRY(kv8_cache(k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens, T, B, Hkv, D, page, num_pages,
                   table_width, max_q_len, c));
  size_t kb = 0, vb = 0;
  MQ_TRY(kv8_rows(k, T, Hkv * D, k_stride, "k", kb));
  MQ_TRY(kv8_rows(v, T, Hkv * D, v_stride, "v", vb));
  const size_t cache = static_cast<size_t>(num_pages) * Hkv * page * D, sc = static_cast<size_t>(num_pages) * Hkv * 4;
  const Range in[] = {{k, kb, "k"},
                      {v, vb, "v"},
                      {block_table, static_cast<size_t>(B * table_width) * 4, "block_table"},
                      {cu_q, static_cast<size_t>(B + 1) * 4, "cu_q"},
                      {kv_lens, static_cast<size_t>(B) * 4, "kv_lens"}};
  const Range out[] = {{k_cache, cache, "k_cache"}, {v_cache, cache, "v_cache"}, {k_scales, sc, "k_scales"}, {v_scales, sc, "v_scales"}};
  MQ_TRY(check_alias(in, out));
  if (T == 0 || B == 0) return ok();
  if (mq::kv8_append_blocks(c) >= (int64_t{1} << 24))
    return fail(MQ_ERR_SHAPE, "B * pages of max_q_len tokens * Hkv = %lld must stay below 2^23",
                (long long)(mq::kv8_append_blocks(c) / 2));
  return hip_status(mq::launch_kv8_append(c, k, v, k_stride, v_stride, bf16, as_stream(stream)), "kv8_append launch");
}

mq_status mq_kv8_append(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride, uint8_t* k_cache,
                        uint8_t* v_cache, float* k_scales, float* v_scales, const int32_t* block_table,
                        const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int64_t B, int64_t Hkv, int64_t D,
                        int64_t page, int64_t num_pages, int64_t table_width, int64_t max_q_len, void* stream) {
  return kv8_append_impl(k, v, k_stride, v_stride, k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens, T, B,
                         Hkv, D, page, num_pages, table_width, max_q_len, false, stream);
}

mq_status mq_kv8_append_bf16(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride, uint8_t* k_cache,
                             uint8_t* v_cache, float* k_scales, float* v_scales, const int32_t* block_table,
                             const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int64_t B, int64_t Hkv, int64_t D,
                             int64_t page, int64_t num_pages, int64_t table_width, int64_t max_q_len, void* stream) {
  return kv8_append_impl(k, v, k_stride, v_stride, k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens, T, B,
                         Hkv, D, page, num_pages, table_width, max_q_len, true, stream);
}

static mq_status kv8_heads(int64_t Hq, int64_t Hkv) {
  if (Hq < 1 || Hq > 1024 || Hkv < 1 || Hq % Hkv)
    return fail(MQ_ERR_SHAPE, "Hq=%lld must be a multiple of Hkv=%lld, at most 1024", (long long)Hq, (long long)Hkv);
  return MQ_OK;
}

// The plan of a call of these sizes; false where it is refused or does nothing.
static bool kv8_plan(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t table_width,
                     int64_t max_q_len, mq::Kv8Plan& plan) {
  // any addresses do: only sizes are looked at
  static const float some[4] = {};
  const uint8_t* const p = reinterpret_cast<const uint8_t*>(16);
  const int32_t* const t = reinterpret_cast<const int32_t*>(some);
  mq::Kv8Cache c;
  if (kv8_cache(p, p, some, some, t, t, t, T, B, Hkv, D, page, 1, table_width, max_q_len, c) != MQ_OK ||
      kv8_heads(Hq, Hkv) != MQ_OK || T == 0 || B == 0)
    return false;
  plan = mq::plan_kv8_attention(c, static_cast<int>(Hq));
  return true;
}

size_t mq_kv8_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page,
                                        int64_t table_width, int64_t max_q_len) {
  mq::Kv8Plan plan;
  return kv8_plan(T, B, Hq, Hkv, D, page, table_width, max_q_len, plan) ? plan.workspace_bytes : 0;
}

int32_t mq_kv8_attention_form(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page,
                              int64_t table_width, int64_t max_q_len) {
  mq::Kv8Plan plan;
  return !kv8_plan(T, B, Hq, Hkv, D, page, table_width, max_q_len, plan) ? MQ_KV8_FORM_NONE
         : plan.decode                                                  ? MQ_KV8_FORM_DECODE
                                                                        : MQ_KV8_FORM_PROMPT;
}

static mq_status kv8_attention_impl(const uint16_t* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                                    const float* k_scales, const float* v_scales, const int32_t* block_table,
                                    const int32_t* cu_q, const int32_t* kv_lens, uint16_t* out, int64_t T, int64_t B,
                                    int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t num_pages,
                                    int64_t table_width, int64_t max_q_len, float softmax_scale, void* workspace,
                                    size_t workspace_bytes, bool bf16, void* stream) {
  mq::Kv8Cache c;
  MQ_TRY(kv8_cache(k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens, T, B, Hkv, D, page, num_pages,
                   table_width, max_q_len, c));
  MQ_TRY(kv8_heads(Hq, Hkv));
  if (!(softmax_scale >= 0.f && softmax_scale <= 1e6f))
    return fail(MQ_ERR_UNSUPPORTED, "softmax_scale=%g must lie in [0, 1e6]", static_cast<double>(softmax_scale));
  size_t qb = 0;
  MQ_TRY(kv8_rows(q, T, Hq * D, q_stride, "q", qb));
  MQ_TRY(need(out, T, "out"));
  if (!aligned(out, 16)) return fail(MQ_ERR_ALIGN, "out must be 16-byte aligned");
  const mq::Kv8Plan plan = mq::plan_kv8_attention(c, static_cast<int>(Hq));
  const bool empty = T == 0 || B == 0;
  const size_t ws = empty ? 0 : plan.workspace_bytes;
  MQ_TRY(check_workspace(workspace, workspace_bytes, ws));
  const size_t cache = static_cast<size_t>(num_pages) * Hkv * page * D, sc = static_cast<size_t>(num_pages) * Hkv * 4;
  const Range in[] = {{q, qb, "q"},
                      {k_cache, cache, "k_cache"},
                      {v_cache, cache, "v_cache"},
                      {k_scales, sc, "k_scales"},
                      {v_scales, sc, "v_scales"},
                      {block_table, static_cast<size_t>(B * table_width) * 4, "block_table"},
                      {cu_q, static_cast<size_t>(B + 1) * 4, "cu_q"},
                      {kv_lens, static_cast<size_t>(B) * 4, "kv_lens"}};
  const Range outs[] = {{out, static_cast<size_t>(T) * Hq * D * 2, "out"}, {ws ? workspace : nullptr, ws, "workspace"}};
  MQ_TRY(check_alias(in, outs));
  if (empty) return ok();
  return hip_status(mq::launch_kv8_attention(c, q, q_stride, out, static_cast<int>(Hq), softmax_scale, plan,
                                             ws ? workspace : nullptr, bf16, as_stream(stream)),
                    "kv8_attention launch");
}

mq_status mq_kv8_attention(const uint16_t* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                           const float* k_scales, const float* v_scales, const int32_t* block_table, const int32_t* cu_q,
                           const int32_t* kv_lens, uint16_t* out, int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                           int64_t page, int64_t num_pages, int64_t table_width, int64_t max_q_len, float softmax_scale,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return kv8_attention_impl(q, q_stride, k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens, out, T, B, Hq,
                            Hkv, D, page, num_pages, table_width, max_q_len, softmax_scale, workspace, workspace_bytes,
                            false, stream);
}

mq_status mq_kv8_attention_bf16(const uint16_t* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                                const float* k_scales, const float* v_scales, const int32_t* block_table,
                                const int32_t* cu_q, const int32_t* kv_lens, uint16_t* out, int64_t T, int64_t B,
                                int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t num_pages, int64_t table_width,
                                int64_t max_q_len, float softmax_scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return kv8_attention_impl(q, q_stride, k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens, out, T, B, Hq,
                            Hkv, D, page, num_pages, table_width, max_q_len, softmax_scale, workspace, workspace_bytes,
                            true, stream);
}

}  // extern "C"
