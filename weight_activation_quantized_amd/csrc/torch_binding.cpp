// Native half of the Python wrappers of the RMS norm, e4m3 and KV-cache entry
// points: the checks of the tensors' metadata, the outputs' allocation and the
// call into libmq, which in Python cost 12-21 us a call, several times what
// the smaller kernels take. Same checks, messages and exceptions as the
// wrappers written in Python; the computation is libmq's alone.
//
// libmq's functions arrive as addresses (bind), so that this module works with
// whichever build of the library the package loaded. Every tensor of a call
// must be on one GPU; outputs are allocated, and the kernels launched, on that
// GPU's current stream.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>

#include "mq.h"

namespace {

struct Library {
  decltype(&mq_rmsnorm_int8) rmsnorm_int8[2];  // fp16, bf16
  decltype(&mq_rmsnorm_fp8) rmsnorm_fp8[2];
  decltype(&mq_quant_fp8_blocks) quant_fp8_blocks[2];
  decltype(&mq_fp8_block_mm_workspace_bytes) fp8_block_mm_workspace_bytes;
  decltype(&mq_fp8_block_mm) fp8_block_mm[2];
  decltype(&mq_fp8_linear_workspace_bytes) fp8_linear_workspace_bytes;
  decltype(&mq_fp8_linear) fp8_linear[2];
  decltype(&mq_kv8_append) kv8_append[2];
  decltype(&mq_kv8_attention_workspace_bytes) kv8_attention_workspace_bytes;
  decltype(&mq_kv8_attention) kv8_attention[2];
} lib;

PyObject* check_fn = nullptr;  // the package's _check(status): raises MqError

// What the wrappers raise for arguments they refuse.
struct Refusal : torch::PyTorchError {
  Refusal(PyObject* type, const char* format, va_list args) : type_(type) {
    char text[512];
    std::vsnprintf(text, sizeof(text), format, args);
    msg = text;
  }
  PyObject* python_type() override { return type_; }
  PyObject* type_;
};
[[noreturn]] __attribute__((format(printf, 1, 2))) void type_error(const char* format, ...) {
  va_list args;
  va_start(args, format);
  const Refusal r(PyExc_TypeError, format, args);
  va_end(args);
  throw r;
}
[[noreturn]] __attribute__((format(printf, 1, 2))) void value_error(const char* format, ...) {
  va_list args;
  va_start(args, format);
  const Refusal r(PyExc_ValueError, format, args);
  va_end(args);
  throw r;
}

std::string shape_text(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}

const char* dtype_text(at::ScalarType d) {
  switch (d) {
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(d);
  }
}

const at::Tensor& any_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error("%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void on_gpu(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) value_error("%s must be on a GPU (got %s)", name, t.device().str().c_str());
}

// A dense tensor of the type and rank on a GPU.
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType dtype, int64_t ndim) {
  const at::Tensor& t = any_tensor(o, name);
  on_gpu(t, name);
  if (t.scalar_type() != dtype)
    type_error("%s must be %s (got %s)", name, dtype_text(dtype), dtype_text(t.scalar_type()));
  if (t.dim() != ndim)
    value_error("%s must be %d-D (got shape %s)", name, static_cast<int>(ndim), shape_text(t).c_str());
  if (!t.is_contiguous()) value_error("%s must be contiguous", name);
  return t;
}

at::ScalarType half_dtype(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) {
    const at::ScalarType d = THPVariable_Unpack(o).scalar_type();
    if (d == at::kHalf || d == at::kBFloat16) return d;
  }
  type_error("%s must be a float16 or bfloat16 tensor", name);
}

void same_device(const at::Tensor& a, const at::Tensor& b) {
  if (a.device() != b.device())
    value_error("tensors on %s and %s: one call takes one GPU's", a.device().str().c_str(),
                            b.device().str().c_str());
}

// The caller's output, checked, or a fresh one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
  const at::Tensor& t = tensor(o, name, dtype, static_cast<int64_t>(shape.size()));
  if (t.sizes() != shape) {
    std::string want = "(";
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    value_error("%s must have shape %s (got %s)", name, (want + (shape.size() == 1 ? ",)" : ")")).c_str(),
                            shape_text(t).c_str());
  }
  same_device(like, t);
  return t;
}

struct Workspace {
  at::Tensor t;
  void* p = nullptr;
  size_t bytes = 0;
};
Workspace workspace(PyObject* o, size_t need, const at::Tensor& like) {
  Workspace w;
  if (o == Py_None) {
    if (need == 0) return w;
    w.t = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(like.device()));
  } else {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda() || !THPVariable_Unpack(o).is_contiguous())
      value_error("workspace must be a contiguous GPU tensor");
    w.t = THPVariable_Unpack(o);
    same_device(like, w.t);
  }
  w.p = w.t.data_ptr();
  w.bytes = w.t.nbytes();
  return w;
}

void* stream_of(const at::Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

// Raises MqError (through the package) for a status that is not MQ_OK.
bool passed(mq_status s) {
  if (s == MQ_OK) return true;
  PyObject* r = PyObject_CallFunction(check_fn, "i", static_cast<int>(s));
  if (r) {
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, "libmq call failed");
  }
  return false;
}

template <typename T>
T* data(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

int64_t blocks(int64_t n) { return (n + 127) / 128; }

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("%s must be an integer", name);
  }
  return v;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("%s must be a number", name);
  }
  return v;
}

#define MQ_ARGS(N)                                                                  \
  if (nargs != (N)) {                                                               \
    PyErr_Format(PyExc_TypeError, "%d arguments needed, %zd given", N, nargs);      \
    return nullptr;                                                                 \
  }

// (x, weight, eps, residual, out, s_out, h_out, fp8)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  MQ_ARGS(8)
  const at::ScalarType dt = half_dtype(a[0], "x");
  const at::Tensor& x = tensor(a[0], "x", dt, 2);
  const at::Tensor& w = tensor(a[1], "weight", dt, 1);
  const double eps = number(a[2], "eps");
  const bool fp8 = a[7] == Py_True, residual = a[3] != Py_None, bf = dt == at::kBFloat16;
  const int64_t M = x.size(0), K = x.size(1);
  if (w.size(0) != K) value_error("weight must be [K]");
  same_device(x, w);
  const uint16_t* rp = nullptr;
  if (residual) {
    const at::Tensor& r = tensor(a[3], "residual", dt, 2);
    if (r.sizes() != x.sizes()) value_error("residual must have x's shape");
    same_device(x, r);
    rp = data<uint16_t>(r);
  } else if (a[6] != Py_None) {
    value_error("h_out needs a residual");
  }
  const c10::DeviceGuard guard(x.device());
  at::Tensor q = output(a[4], "out", {M, K}, fp8 ? at::kFloat8_e4m3fn : at::kChar, x);
  at::Tensor s = fp8 ? output(a[5], "s_out", {blocks(K), M}, at::kFloat, x) : output(a[5], "s_out", {M}, at::kFloat, x);
  at::Tensor h;
  if (residual) h = output(a[6], "h_out", {M, K}, dt, x);
  uint16_t* const hp = residual ? data<uint16_t>(h) : nullptr;
  const mq_status st =
      fp8 ? lib.rmsnorm_fp8[bf](data<uint16_t>(x), rp, data<uint16_t>(w), eps, hp, data<uint8_t>(q), data<float>(s), M, K,
                                stream_of(x))
          : lib.rmsnorm_int8[bf](data<uint16_t>(x), rp, data<uint16_t>(w), eps, hp, data<int8_t>(q), data<float>(s), M, K,
                                 stream_of(x));
  if (!passed(st)) return nullptr;
  PyObject* r = PyTuple_New(residual ? 3 : 2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(q)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(s)));
  if (residual) PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(h)));
  return r;
  END_HANDLE_TH_ERRORS
}

// (x, out, s_out)
PyObject* quant_fp8_blocks(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  MQ_ARGS(3)
  const at::ScalarType dt = half_dtype(a[0], "x");
  const at::Tensor& x = tensor(a[0], "x", dt, 2);
  const int64_t M = x.size(0), K = x.size(1);
  const c10::DeviceGuard guard(x.device());
  at::Tensor q = output(a[1], "out", {M, K}, at::kFloat8_e4m3fn, x);
  at::Tensor s = output(a[2], "s_out", {blocks(K), M}, at::kFloat, x);
  if (!passed(lib.quant_fp8_blocks[dt == at::kBFloat16](data<uint16_t>(x), data<uint8_t>(q), data<float>(s), M, K,
                                                        stream_of(x))))
    return nullptr;
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(q)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(s)));
  return r;
  END_HANDLE_TH_ERRORS
}

// wq [N, K], s_w [ceil(N/128), ceil(K/128)]: N.
int64_t fp8_weights(const at::Tensor& wq, const at::Tensor& s_w, int64_t K) {
  const int64_t N = wq.size(0);
  if (wq.size(1) != K || s_w.size(0) != blocks(N) || s_w.size(1) != blocks(K))
    value_error("wq must be [N, K] and s_w [ceil(N/128), ceil(K/128)]");
  same_device(wq, s_w);
  return N;
}

// (xq, s_x, wq, s_w, out, workspace, bf16)
PyObject* fp8_block_mm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  MQ_ARGS(7)
  const at::Tensor& xq = tensor(a[0], "xq", at::kFloat8_e4m3fn, 2);
  const at::Tensor& s_x = tensor(a[1], "s_x", at::kFloat, 2);
  const at::Tensor& wq = tensor(a[2], "wq", at::kFloat8_e4m3fn, 2);
  const at::Tensor& s_w = tensor(a[3], "s_w", at::kFloat, 2);
  const bool bf = a[6] == Py_True;
  const int64_t M = xq.size(0), K = xq.size(1);
  if (s_x.size(0) != blocks(K) || s_x.size(1) != M) value_error("s_x must be [ceil(K/128), M]");
  const int64_t N = fp8_weights(wq, s_w, K);
  same_device(xq, s_x);
  same_device(xq, wq);
  const c10::DeviceGuard guard(xq.device());
  at::Tensor y = output(a[4], "out", {M, N}, bf ? at::kBFloat16 : at::kHalf, xq);
  const Workspace w = workspace(a[5], lib.fp8_block_mm_workspace_bytes(M, N, K), xq);
  if (!passed(lib.fp8_block_mm[bf](data<uint8_t>(xq), data<float>(s_x), data<uint8_t>(wq), data<float>(s_w),
                                   data<uint16_t>(y), M, N, K, w.p, w.bytes, stream_of(xq))))
    return nullptr;
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// (x, wq, s_w, out, workspace)
PyObject* fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  MQ_ARGS(5)
  const at::ScalarType dt = half_dtype(a[0], "x");
  const at::Tensor& x = tensor(a[0], "x", dt, 2);
  const at::Tensor& wq = tensor(a[1], "wq", at::kFloat8_e4m3fn, 2);
  const at::Tensor& s_w = tensor(a[2], "s_w", at::kFloat, 2);
  const int64_t M = x.size(0), K = x.size(1), N = fp8_weights(wq, s_w, K);
  same_device(x, wq);
  const c10::DeviceGuard guard(x.device());
  at::Tensor y = output(a[3], "out", {M, N}, dt, x);
  const Workspace w = workspace(a[4], lib.fp8_linear_workspace_bytes(M, N, K), x);
  if (!passed(lib.fp8_linear[dt == at::kBFloat16](data<uint16_t>(x), data<uint8_t>(wq), data<float>(s_w),
                                                  data<uint16_t>(y), M, N, K, w.p, w.bytes, stream_of(x))))
    return nullptr;
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// Rows [T, heads, D] of a 16-bit tensor, dense within a row: their stride in values.
int64_t kv8_rows(const at::Tensor& t, const char* name, at::ScalarType dtype, int64_t D) {
  if (t.scalar_type() != dtype) type_error("%s must be a %s tensor", name, dtype_text(dtype));
  on_gpu(t, name);
  if (t.dim() != 3 || t.size(2) != D)
    value_error("%s must be [T, heads, %lld] (got shape %s)", name, static_cast<long long>(D),
                            shape_text(t).c_str());
  const int64_t T = t.size(0), H = t.size(1);
  if (T == 0) return H * D;
  if (t.stride(2) != 1 || (H > 1 && t.stride(1) != D))
    value_error("%s: a token's heads must lie side by side", name);
  return T > 1 ? t.stride(0) : H * D;
}

struct Cache {
  const at::Tensor &k, &v, &ks, &vs, &table, &cu, &lens;
  int64_t P, H, page, D, B, width;
};

// k_cache, v_cache, k_scales, v_scales, block_table, cu_q, kv_lens
Cache kv8_cache(PyObject* const* a) {
  Cache c = {tensor(a[0], "k_cache", at::kFloat8_e4m3fn, 4), tensor(a[1], "v_cache", at::kFloat8_e4m3fn, 4),
             tensor(a[2], "k_scales", at::kFloat, 2),        tensor(a[3], "v_scales", at::kFloat, 2),
             tensor(a[4], "block_table", at::kInt, 2),       tensor(a[5], "cu_q", at::kInt, 1),
             tensor(a[6], "kv_lens", at::kInt, 1),           0, 0, 0, 0, 0, 0};
  c.P = c.k.size(0);
  c.H = c.k.size(1);
  c.page = c.k.size(2);
  c.D = c.k.size(3);
  if (c.v.sizes() != at::IntArrayRef({c.P, c.H, c.D, c.page}))
    value_error("k_cache must be [P, Hkv, page, D] and v_cache [P, Hkv, D, page]");
  if (c.ks.sizes() != at::IntArrayRef({c.P, c.H}) || c.vs.sizes() != at::IntArrayRef({c.P, c.H}))
    value_error("k_scales and v_scales must be [P, Hkv]");
  c.B = c.table.size(0);
  c.width = c.table.size(1);
  if (c.cu.size(0) != c.B + 1 || c.lens.size(0) != c.B)
    value_error("cu_q must be [B + 1] and kv_lens [B] for block_table [B, width]");
  for (const at::Tensor* t : {&c.v, &c.ks, &c.vs, &c.table, &c.cu, &c.lens}) same_device(c.k, *t);
  return c;
}

// (k, v, the cache's seven, max_q_len)
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  MQ_ARGS(10)
  const at::ScalarType dt = half_dtype(a[0], "k");
  const Cache c = kv8_cache(a + 2);
  const at::Tensor &k = any_tensor(a[0], "k"), &v = any_tensor(a[1], "v");
  const int64_t ks = kv8_rows(k, "k", dt, c.D), vs = kv8_rows(v, "v", dt, c.D);
  if (k.sizes() != v.sizes() || k.size(1) != c.H) value_error("k and v must be [T, Hkv, D]");
  same_device(c.k, k);
  same_device(c.k, v);
  const int64_t most = integer(a[9], "max_q_len");
  const c10::DeviceGuard guard(c.k.device());
  if (!passed(lib.kv8_append[dt == at::kBFloat16](
          data<uint16_t>(k), data<uint16_t>(v), ks, vs, data<uint8_t>(c.k), data<uint8_t>(c.v), data<float>(c.ks),
          data<float>(c.vs), data<int32_t>(c.table), data<int32_t>(c.cu), data<int32_t>(c.lens), k.size(0), c.B, c.H,
          c.D, c.page, c.P, c.width, most, stream_of(c.k))))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (q, the cache's seven, max_q_len, softmax_scale, out, workspace)
PyObject* kv8_attention(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  MQ_ARGS(12)
  const at::ScalarType dt = half_dtype(a[0], "q");
  const Cache c = kv8_cache(a + 1);
  const at::Tensor& q = any_tensor(a[0], "q");
  const int64_t qs = kv8_rows(q, "q", dt, c.D);
  const int64_t T = q.size(0), Hq = q.size(1), most = integer(a[8], "max_q_len");
  const float scale = static_cast<float>(a[9] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.D))
                                                         : number(a[9], "softmax_scale"));
  same_device(q, c.k);
  const c10::DeviceGuard guard(q.device());
  at::Tensor o = output(a[10], "out", {T, Hq, c.D}, dt, q);
  const Workspace w =
      workspace(a[11], lib.kv8_attention_workspace_bytes(T, c.B, Hq, c.H, c.D, c.page, c.width, most), q);
  if (!passed(lib.kv8_attention[dt == at::kBFloat16](
          data<uint16_t>(q), qs, data<uint8_t>(c.k), data<uint8_t>(c.v), data<float>(c.ks), data<float>(c.vs),
          data<int32_t>(c.table), data<int32_t>(c.cu), data<int32_t>(c.lens), data<uint16_t>(o), T, c.B, Hq, c.H, c.D,
          c.page, c.P, c.width, most, scale, w.p, w.bytes, stream_of(q))))
    return nullptr;
  return THPVariable_Wrap(std::move(o));
  END_HANDLE_TH_ERRORS
}

// bind(addresses in the order of Library, check): once, when the package loads libmq.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  MQ_ARGS(2)
  constexpr size_t kCount = sizeof(Library) / sizeof(void*);
  if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != static_cast<Py_ssize_t>(kCount)) {
    PyErr_Format(PyExc_ValueError, "bind needs %zu addresses", kCount);
    return nullptr;
  }
  void* at[kCount];
  for (size_t i = 0; i < kCount; ++i) {
    at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
    if (PyErr_Occurred()) return nullptr;
    if (!at[i]) {
      PyErr_SetString(PyExc_ValueError, "bind: a NULL address");
      return nullptr;
    }
  }
  static_assert(sizeof(Library) == sizeof(at), "Library holds function pointers only");
  std::memcpy(&lib, at, sizeof(at));
  Py_INCREF(a[1]);
  Py_XSETREF(check_fn, a[1]);
  Py_RETURN_NONE;
}

#define MQ_METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MQ_METHOD(bind),       MQ_METHOD(rmsnorm),    MQ_METHOD(quant_fp8_blocks),
                         MQ_METHOD(fp8_block_mm), MQ_METHOD(fp8_linear), MQ_METHOD(kv8_append),
                         MQ_METHOD(kv8_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mq_torch", "Native half of the package's torch wrappers.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mq_torch(void) { return PyModule_Create(&module); }
