// Python binding of the operators around a layer's products, as one extension
// module (moe_expert_gb300._native): argument checks, output allocation and the
// call of the C entry point in C++.  Called once a token and layer, these calls
// cost less on the GPU than their marshalling did in Python: a call with three
// outputs took 17 us through ctypes and torch.empty on the host of a GB300.
// Every step of the computation is behind the C ABI (include/moex.h).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/moex.h"

namespace {

PyObject* g_error_class = nullptr;  // MoexError, set by the package

struct TypeRefused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // a Python exception is set already

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw TypeRefused(std::string(what) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

std::optional<at::Tensor> maybe(PyObject* o, const char* what) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, what);
}

int64_t integer(PyObject* o, int64_t lo, int64_t hi, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  if (v < lo || v > hi) refuse(std::string(what) + ": out of range");
  return v;
}
int int32(PyObject* o, const char* what) {
  return static_cast<int>(integer(o, INT32_MIN, INT32_MAX, what));
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v != 0;
}

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return MOEX_F32;
    case at::kBFloat16: return MOEX_BF16;
    case at::kHalf: return MOEX_F16;
    default: throw TypeRefused("expected float32, bfloat16 or float16");
  }
}

std::optional<at::ScalarType> maybe_dtype(PyObject* o) {
  if (o == Py_None) return std::nullopt;
  if (!THPDtype_Check(o)) throw TypeRefused("expected a torch dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int32_t count(int64_t n, const char* what) {
  if (n > INT32_MAX) refuse(std::string(what) + ": too large");
  return static_cast<int32_t>(n);
}

// Row stride of a matrix of rows x width with contiguous rows (the width for a
// single row, whose stride says nothing).
int64_t row_stride(const at::Tensor& t, int64_t rows, int64_t width, const char* what) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != width || (width > 1 && t.stride(1) != 1))
    refuse(std::string(what) + ": expected [" + std::to_string(rows) + ", " + std::to_string(width) +
           "], rows contiguous");
  return rows > 1 ? t.stride(0) : width;
}

void* flat(const at::Tensor& t, int64_t numel, at::ScalarType type, const char* what) {
  if (t.numel() != numel || t.scalar_type() != type || !t.is_contiguous())
    refuse(std::string(what) + ": expected " + std::to_string(numel) + " contiguous elements of " +
           c10::toString(type));
  return t.data_ptr();
}

// Token stride of [tokens][heads][dim] with contiguous tokens.
int64_t token_stride(const at::Tensor& t, int64_t tokens, int64_t heads, int64_t dim, const char* what) {
  if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim || t.stride(2) != 1 ||
      (heads > 1 && t.stride(1) != dim))
    refuse(std::string(what) + ": expected [" + std::to_string(tokens) + ", " + std::to_string(heads) + ", " +
           std::to_string(dim) + "], heads contiguous");
  return tokens > 1 ? t.stride(0) : heads * dim;
}

at::Tensor fresh(at::IntArrayRef size, const at::Tensor& like, at::ScalarType type) {
  return at::empty(size, like.options().dtype(type));
}

// The device of a call, current while this lives: the launch, the allocations and
// the status word are that device's, whichever was current.  Every tensor among
// the call's arguments has to be on it.
class CallDevice {
 public:
  CallDevice(PyObject* const* a, Py_ssize_t n, const at::Tensor& first) {
    const at::Device device = first.device();
    for (Py_ssize_t i = 0; i < n; ++i) {
      // what is plainly no tensor first: for those the check itself is a slow one
      if (a[i] == Py_None || PyLong_Check(a[i]) || PyFloat_Check(a[i]) || THPDtype_Check(a[i]) ||
          !THPVariable_Check(a[i]))
        continue;
      const at::Tensor& t = THPVariable_Unpack(a[i]);
      if (!t.is_cuda()) refuse("every tensor has to be a CUDA tensor");
      if (t.device() != device)
        refuse("every tensor has to be on one device: " + device.str() + " and " + t.device().str());
    }
    if (c10::cuda::current_device() != device.index()) guard_.set_device(device);
  }

 private:
  c10::cuda::OptionalCUDAGuard guard_;
};

// The stream of a call on that device: the handle in the last argument, else
// torch's current one.  What is allocated while this lives belongs to that stream,
// so a workspace that is released when the call returns is not handed to another
// stream's tensor while the kernels still use it.
class CallStream {
 public:
  CallStream(PyObject* const* a, Py_ssize_t n, const at::Tensor& first) : device_(a, n, first) {
    PyObject* const o = a[n - 1];
    const auto index = first.device().index();
    handle_ = c10::cuda::getCurrentCUDAStream(index).stream();
    if (o == Py_None) return;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError();
    const cudaStream_t given = static_cast<cudaStream_t>(p);
    if (given == handle_) return;
    handle_ = given;
    guard_.emplace(handle_ ? c10::cuda::getStreamFromExternal(handle_, index) : c10::cuda::getDefaultCUDAStream(index));
  }
  operator moex_stream() const { return reinterpret_cast<moex_stream>(handle_); }

 private:
  CallDevice device_;
  cudaStream_t handle_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

void check(moex_status st, const char* what) {
  if (st == MOEX_OK) return;
  PyObject* e = g_error_class ? PyObject_CallFunction(g_error_class, "is", static_cast<int>(st), what) : nullptr;
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "%s: %s", what, moex_status_string(st));
  }
  throw PythonError();
}

PyObject* wrap(const std::optional<at::Tensor>& t) {
  if (!t) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}

// No C++ exception leaves a function that Python calls.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, want, got);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const PythonError&) {
    return nullptr;
  } catch (const TypeRefused& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (x, gamma, eps, residual, sum_out, y, y_dtype, quantize, q, ds, stream) -> (sum_out, y, q, ds)
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("add_rms_norm", n, 11, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& gamma = tensor(a[1], "gamma");
    const CallStream stream(a, n, x);
    if (x.dim() != 2) refuse("x: expected [T, H]");
    const int64_t T = x.size(0), H = x.size(1);
    const int64_t ldx = row_stride(x, T, H, "x");
    const int xt = type_code(x.scalar_type());
    auto residual = maybe(a[3], "residual"), sum = maybe(a[4], "sum_out"), y = maybe(a[5], "y"), q = maybe(a[8], "q"),
         ds = maybe(a[9], "ds");
    const auto y_dtype = maybe_dtype(a[6]);
    int64_t ldr = 0, lds = 0, ldy = 0;
    if (residual) {
      ldr = row_stride(*residual, T, H, "residual");
      if (residual->scalar_type() != at::kFloat) refuse("residual: expected float32");
      if (!sum) sum = fresh({T, H}, x, at::kFloat);
    }
    if (sum) {
      lds = row_stride(*sum, T, H, "sum_out");
      if (sum->scalar_type() != at::kFloat) refuse("sum_out: expected float32");
    }
    if (!y && y_dtype) y = fresh({T, H}, x, *y_dtype);
    if (y) ldy = row_stride(*y, T, H, "y");
    int8_t* qp = nullptr;
    float* dp = nullptr;
    if (truth(a[7])) {
      if (!q) q = fresh({T, H}, x, at::kChar);
      if (!ds) ds = fresh({T, H / 32, 2}, x, at::kFloat);
      qp = static_cast<int8_t*>(flat(*q, T * H, at::kChar, "q"));
      dp = static_cast<float*>(flat(*ds, T * (H / 32) * 2, at::kFloat, "ds"));
    } else {
      q = ds = std::nullopt;
    }
    check(moex_add_rms_norm(x.data_ptr(), xt, ldx, residual ? residual->data_ptr<float>() : nullptr, ldr,
                            static_cast<float*>(flat(gamma, H, at::kFloat, "gamma")), static_cast<float>(real(a[2])),
                            count(T, "T"), H, sum ? sum->data_ptr<float>() : nullptr, lds, y ? y->data_ptr() : nullptr,
                            y ? type_code(y->scalar_type()) : MOEX_F32, ldy, qp, dp, stream),
          "moex_add_rms_norm");
    PyObject* r = PyTuple_New(4);
    if (!r) throw PythonError();
    PyTuple_SET_ITEM(r, 0, wrap(sum));
    PyTuple_SET_ITEM(r, 1, wrap(y));
    PyTuple_SET_ITEM(r, 2, wrap(q));
    PyTuple_SET_ITEM(r, 3, wrap(ds));
    return r;
  });
}

// (q, ds, y, dtype, stream) -> y
PyObject* dequantize_q8_1(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("dequantize_q8_1", n, 5, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor& ds = tensor(a[1], "ds");
    const CallStream stream(a, n, q);
    if (q.dim() != 2) refuse("q: expected [T, K]");
    const int64_t T = q.size(0), K = q.size(1);
    auto y = maybe(a[2], "y");
    const auto dtype = maybe_dtype(a[3]);
    void* qp = flat(q, T * K, at::kChar, "q");
    void* dp = flat(ds, T * (K / 32) * 2, at::kFloat, "ds");
    if (!y) y = fresh({T, K}, q, dtype.value_or(at::kFloat));
    check(moex_dequantize_q8_1(static_cast<int8_t*>(qp), static_cast<float*>(dp), count(T, "T"), K,
                               flat(*y, T * K, y->scalar_type(), "y"), type_code(y->scalar_type()),
                               stream),
          "moex_dequantize_q8_1");
    return wrap(y);
  });
}

// (logits, k, score, bias, groups, top_groups, group_top, renorm, scale, ids, w, stream) -> (ids, w)
PyObject* route_experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("route_experts", n, 12, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "logits");
    const CallStream stream(a, n, x);
    if (x.dim() != 2) refuse("logits: expected [T, E]");
    const int64_t T = x.size(0), E = x.size(1);
    const int64_t ldl = row_stride(x, T, E, "logits");
    const int k = int32(a[1], "k");
    auto bias = maybe(a[3], "bias"), ids = maybe(a[9], "ids"), w = maybe(a[10], "w");
    if (k < 1) check(MOEX_EINVAL, "moex_route_experts");
    if (!ids) ids = fresh({T, k}, x, at::kInt);
    if (!w) w = fresh({T, k}, x, at::kFloat);
    check(moex_route_experts(x.data_ptr(), type_code(x.scalar_type()), ldl,
                             bias ? static_cast<float*>(flat(*bias, E, at::kFloat, "bias")) : nullptr, count(T, "T"),
                             count(E, "E"), k, int32(a[2], "score"), int32(a[4], "groups"), int32(a[5], "top_groups"),
                             int32(a[6], "group_top"), truth(a[7]) ? 1 : 0, static_cast<float>(real(a[8])),
                             static_cast<int32_t*>(flat(*ids, T * k, at::kInt, "ids")),
                             static_cast<float*>(flat(*w, T * k, at::kFloat, "w")), stream),
          "moex_route_experts");
    PyObject* r = PyTuple_New(2);
    if (!r) throw PythonError();
    PyTuple_SET_ITEM(r, 0, wrap(ids));
    PyTuple_SET_ITEM(r, 1, wrap(w));
    return r;
  });
}

moex_paged_kv paged_kv(PyObject* ko, PyObject* vo) {
  const at::Tensor& k = tensor(ko, "k_cache");
  const at::Tensor& v = tensor(vo, "v_cache");
  if (k.dim() != 4 || v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes() || v.strides() != k.strides() ||
      k.stride(3) != 1)
    refuse("k_cache and v_cache: the same type, shape [pages, heads, page, dim] and strides, dim contiguous");
  moex_paged_kv kv;
  kv.type = type_code(k.scalar_type());
  kv.n_pages = k.size(0);
  kv.n_kv_heads = count(k.size(1), "key heads");
  kv.page_size = count(k.size(2), "page size");
  kv.head_dim = count(k.size(3), "head size");
  kv.page_stride = k.stride(0);
  kv.head_stride = k.stride(1);
  kv.row_stride = k.stride(2);
  kv.k = k.data_ptr();
  kv.v = v.data_ptr();
  return kv;
}

// cu_q, ctx_len, page_table at a[0 .. 2]
moex_batch batch_of(PyObject* const* a, int64_t tokens, PyObject* max_q) {
  const at::Tensor& cu = tensor(a[0], "cu_q");
  const at::Tensor& ctx = tensor(a[1], "ctx_len");
  const at::Tensor& table = tensor(a[2], "page_table");
  if (table.dim() != 2 || table.scalar_type() != at::kInt || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("page_table: expected int32 [B, width], rows contiguous");
  moex_batch b;
  const int64_t n = table.size(0);
  b.n_seqs = count(n, "sequences");
  b.n_tokens = count(tokens, "tokens");
  // without a hint, the most that sequences of one token or more can have: single tokens are seen as such
  if (max_q == nullptr || max_q == Py_None)
    b.max_q = b.n_tokens < b.n_seqs ? b.n_tokens : b.n_tokens - b.n_seqs + 1;
  else
    b.max_q = int32(max_q, "max_q");
  b.table_width = count(table.size(1), "page table width");
  b.table_stride = n > 1 ? table.stride(0) : table.size(1);
  b.cu_q = static_cast<int32_t*>(flat(cu, n + 1, at::kInt, "cu_q"));
  b.ctx_len = static_cast<int32_t*>(flat(ctx, n, at::kInt, "ctx_len"));
  b.page_table = static_cast<int32_t*>(table.data_ptr());
  return b;
}

// (qkv, k_cache, v_cache, cu_q, ctx_len, page_table, n_heads, cos_sin, interleaved, q, stream) -> q
PyObject* rope_kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rope_kv_write", n, 11, [&]() -> PyObject* {
    const at::Tensor& qkv = tensor(a[0], "qkv");
    const CallStream stream(a, n, qkv);
    if (qkv.dim() != 2) refuse("qkv: expected [T, (n_heads + 2 * kv_heads) * dim]");
    const int64_t T = qkv.size(0);
    const moex_paged_kv kv = paged_kv(a[1], a[2]);
    const moex_batch b = batch_of(a + 3, T, nullptr);
    const int heads = int32(a[6], "n_heads");
    const int64_t D = kv.head_dim;
    const int64_t ld = row_stride(qkv, T, (heads + 2 * static_cast<int64_t>(kv.n_kv_heads)) * D, "qkv");
    auto cs = maybe(a[7], "cos_sin"), q = maybe(a[9], "q");
    int64_t n_pos = 0, rot = 0;
    const float* csp = nullptr;
    if (cs) {
      if (cs->dim() != 2) refuse("cos_sin: expected float32 [positions, rot_dim]");
      n_pos = cs->size(0);
      rot = cs->size(1);
      csp = static_cast<float*>(flat(*cs, n_pos * rot, at::kFloat, "cos_sin"));
    }
    const at::ScalarType ct = THPVariable_Unpack(a[1]).scalar_type();
    if (heads < 1) check(MOEX_EINVAL, "moex_rope_kv_write");
    if (!q) q = fresh({T, heads, D}, qkv, ct);
    if (q->scalar_type() != ct) refuse("q: expected the cache's type");
    check(moex_rope_kv_write(qkv.data_ptr(), type_code(qkv.scalar_type()), ld, &kv, &b, heads, csp, n_pos,
                             count(rot, "rot_dim"), truth(a[8]) ? 1 : 0, q->data_ptr(),
                             token_stride(*q, T, heads, D, "q"), stream),
          "moex_rope_kv_write");
    return wrap(q);
  });
}

// (k_cache, v_cache, cu_q, ctx_len, page_table, n_tokens, n_heads, max_q) -> bytes
PyObject* paged_attention_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention_workspace_bytes", n, 8, [&]() -> PyObject* {
    const CallDevice device(a, n, tensor(a[0], "k_cache"));
    const moex_paged_kv kv = paged_kv(a[0], a[1]);
    const moex_batch b = batch_of(a + 2, int32(a[5], "n_tokens"), a[7]);
    return PyLong_FromSize_t(moex_paged_attention_workspace_bytes(&kv, &b, int32(a[6], "n_heads")));
  });
}

// (q, k_cache, v_cache, cu_q, ctx_len, page_table, max_q, scale, window, out, out_dtype, lse, ws, stream) -> out
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention", n, 14, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const CallStream stream(a, n, q);
    if (q.dim() != 3) refuse("q: expected [T, n_heads, dim]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    const moex_paged_kv kv = paged_kv(a[1], a[2]);
    const moex_batch b = batch_of(a + 3, T, a[6]);
    if (q.scalar_type() != THPVariable_Unpack(a[1]).scalar_type() || D != kv.head_dim)
      refuse("q: expected the cache's type and head size");
    const int64_t ldq = token_stride(q, T, H, D, "q");
    const float scale = a[7] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                        : static_cast<float>(real(a[7]));
    auto out = maybe(a[9], "out"), lse = maybe(a[11], "lse"), ws = maybe(a[12], "ws");
    const auto out_dtype = maybe_dtype(a[10]);
    if (!out) out = fresh({T, H, D}, q, out_dtype.value_or(q.scalar_type()));
    const int64_t ldo = token_stride(*out, T, H, D, "out");
    const int heads = count(H, "n_heads");
    if (!ws) {
      const size_t need = moex_paged_attention_workspace_bytes(&kv, &b, heads);
      if (need) ws = fresh({static_cast<int64_t>(need)}, q, at::kByte);
    }
    const size_t bytes = ws ? static_cast<size_t>(ws->numel()) : 0;
    check(moex_paged_attention(q.data_ptr(), ldq, &kv, &b, heads, scale, int32(a[8], "window"), out->data_ptr(),
                               type_code(out->scalar_type()), ldo,
                               lse ? static_cast<float*>(flat(*lse, T * H, at::kFloat, "lse")) : nullptr,
                               ws ? flat(*ws, static_cast<int64_t>(bytes), at::kByte, "ws") : nullptr, bytes,
                               stream),
          "moex_paged_attention");
    return wrap(out);
  });
}

PyObject* set_error_class(PyObject*, PyObject* c) {
  Py_INCREF(c);
  Py_XSETREF(g_error_class, c);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(add_rms_norm),
                         FAST(dequantize_q8_1),
                         FAST(route_experts),
                         FAST(rope_kv_write),
                         FAST(paged_attention),
                         FAST(paged_attention_workspace_bytes),
                         {"set_error_class", set_error_class, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
