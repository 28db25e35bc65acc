// binding.cpp -- the Python side of the calls that a serving process makes once
// a layer and token (tg_paged_append, tg_paged_attn, tg_quantize_rows,
// tg_linear_quantized). Their kernels take a few microseconds; checking a dozen
// tensors and allocating the results from Python takes longer than that, so it
// is done here: the checks, the allocation through torch, the call of the C ABI
// on torch's current stream (or the given one) with the tensors' device current.
// A check that fails raises ValueError; a status that is not TG_OK is returned
// as an integer, for the caller to raise.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>
#include <optional>
#include <string>

#include "tokengate.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(const std::string& what) {
  throw c10::ValueError({__func__, __FILE__, static_cast<uint32_t>(__LINE__)}, what);
}

const Tensor& need_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// None: no tensor
const Tensor* maybe_tensor(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &need_tensor(o, name);
}

// Sizes that the C ABI holds in 32 bits.
int32_t int32_of(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + " " + std::to_string(n) + " is above 2^31 - 1");
  return static_cast<int32_t>(n);
}

std::string at_device(int64_t index) { return " on cuda:" + std::to_string(index); }
const char* type_name(at::ScalarType t) { return c10::toString(t); }

int64_t cuda_index(const Tensor& t) {
  if (!t.is_cuda()) refuse("tensors must be on a CUDA device");
  return t.get_device();
}

// Pointer of an optional contiguous tensor of n elements.
template <typename P>
const P* vec(const Tensor* t, int64_t n, at::ScalarType type, int64_t index, const char* name) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type || !t->is_cuda() || t->get_device() != index || t->numel() != n ||
      !t->is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + type_name(type) + " tensor of " +
           std::to_string(n) + " elements" + at_device(index));
  return static_cast<const P*>(t->data_ptr());
}

// Row stride of a [rows, heads, dh] tensor whose rows are contiguous.
int64_t rows3(const Tensor& t, int64_t rows, int64_t heads, int64_t dh, at::ScalarType type,
              int64_t index, const char* name) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != index || t.dim() != 3 ||
      t.size(0) != rows || t.size(1) != heads || t.size(2) != dh)
    refuse(std::string(name) + " must be " + type_name(type) + " [" + std::to_string(rows) + ", " +
           std::to_string(heads) + ", " + std::to_string(dh) + "]" + at_device(index));
  if (rows == 0) return heads * dh;
  if (t.stride(2) != 1 || (t.stride(1) != dh && heads != 1))
    refuse(std::string(name) + ": each row must be contiguous");
  return rows > 1 ? t.stride(0) : std::max(t.stride(0), heads * dh);
}

tg_dtype dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return TG_BF16;
  if (t.scalar_type() == at::kFloat) return TG_F32;
  refuse(std::string("unsupported dtype ") + type_name(t.scalar_type()) + " (bf16 or fp32)");
}

// None: the device's current stream; else the stream's handle.
tg_stream stream_of(PyObject* o, int64_t index) {
  if (o == Py_None)
    return reinterpret_cast<tg_stream>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
  return reinterpret_cast<tg_stream>(PyLong_AsVoidPtr(o));
}

// While it lives, what is allocated belongs to the stream of the call: memory
// of the current stream may still be in use there by what was freed last, which
// the caller has no reason to wait for. The results go back to a caller on the
// current stream, so their memory is not to be handed out again before what
// that stream has been given by then is done.
class OnStream {
 public:
  OnStream(PyObject* stream, tg_stream st, int64_t index) {
    if (stream == Py_None) return;
    const auto device = static_cast<c10::DeviceIndex>(index);
    caller_ = c10::cuda::getCurrentCUDAStream(device);
    guard_.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(st), device));
  }
  void result(const Tensor& t) const {
    if (caller_ && t.numel() > 0) t.record_stream(*caller_);
  }

 private:
  std::optional<c10::cuda::CUDAStream> caller_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

// A given output tensor, or a new one: contiguous, of these sizes.
Tensor output(PyObject* o, at::IntArrayRef sizes, at::ScalarType type, int64_t index, const char* what,
              const OnStream& on) {
  if (o == Py_None) {
    Tensor t = at::empty(sizes, at::TensorOptions().dtype(type).device(
                                    c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(index))));
    on.result(t);
    return t;
  }
  const Tensor& t = need_tensor(o, "an output");
  if (t.sizes() != sizes || t.scalar_type() != type || !t.is_cuda() || t.get_device() != index ||
      !t.is_contiguous())
    refuse(what);
  return t;
}

// Runs the call with the device current; the result, or the status as an int.
template <typename F>
PyObject* finish(int64_t index, const F& call, PyObject* (*wrap)(const Tensor*, const Tensor*),
                 const Tensor* r0, const Tensor* r1) {
  tg_status status;
  if (c10::cuda::current_device() == index) {
    status = call();
  } else {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    status = call();
  }
  if (status != TG_OK) return PyLong_FromLong(status);
  return wrap(r0, r1);
}
PyObject* wrap_one(const Tensor* r, const Tensor*) {
  if (r == nullptr) Py_RETURN_NONE;
  return THPVariable_Wrap(*r);
}
PyObject* wrap_two(const Tensor* a, const Tensor* b) {
  PyObject* pair = PyTuple_New(2);
  if (pair == nullptr) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(*a));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(*b));
  return pair;
}

bool arity(Py_ssize_t have, Py_ssize_t want) {
  if (have == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, have);
  return false;
}

// ------------------------------------------------------------------ cache
struct Cache {
  tg_paged_kv c;
  int64_t index;
  int32_t batch;
  at::ScalarType type;
  Tensor k, v, table, bias;  // the memory that c points at
};
constexpr const char* kCache = "tokengate.paged_kv";

void free_cache(PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, kCache)); }

// cache(address of a tg_paged_kv, device index, batch, k, v, table, bias or None): a
// copy of it for the calls, which keeps the tensors
PyObject* make_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 7)) return nullptr;
  const auto* c = static_cast<const tg_paged_kv*>(PyLong_AsVoidPtr(a[0]));
  const long index = PyLong_AsLong(a[1]);
  const long long batch = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  auto* k = new Cache{*c, index, int32_of(batch, "the table's batch"), c->dtype == TG_BF16 ? at::kBFloat16 : at::kFloat,
                      need_tensor(a[3], "k"), need_tensor(a[4], "v"), need_tensor(a[5], "table"),
                      a[6] == Py_None ? Tensor() : need_tensor(a[6], "bias")};
  PyObject* o = PyCapsule_New(k, kCache, free_cache);
  if (o == nullptr) delete k;
  return o;
  END_HANDLE_TH_ERRORS
}

const Cache& cache_of(PyObject* o) {
  const auto* k = static_cast<const Cache*>(PyCapsule_GetPointer(o, kCache));
  if (k == nullptr) throw python_error();
  if (k->index < 0) refuse("tensors must be on a CUDA device");
  return *k;
}

// (cache, k, v, cu_q, kv_len, q, pos, s, q_norm, k_norm, eps, rope_base, q_out, stream)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 14)) return nullptr;
  const Cache& c = cache_of(a[0]);
  const Tensor& k = need_tensor(a[1], "k");
  const Tensor& v = need_tensor(a[2], "v");
  if (k.dim() != 3) refuse("k must be [rows, heads, head_dim]");
  const int64_t rows = k.size(0), hkv = c.c.n_heads_kv, dh = c.c.head_dim, index = c.index;
  const tg_stream st = stream_of(a[13], index);
  if (PyErr_Occurred()) return nullptr;
  const OnStream on(a[13], st, index);
  const int64_t k_st = rows3(k, rows, hkv, dh, c.type, index, "k");
  const int64_t v_st = rows3(v, rows, hkv, dh, c.type, index, "v");
  const Tensor* q = maybe_tensor(a[5], "q");
  int32_t hq = 0;
  int64_t q_st = 0;
  Tensor out;
  if (q != nullptr) {
    if (q->dim() != 3) refuse("q must be [rows, heads, head_dim]");
    hq = int32_of(q->size(1), "q's heads");
    q_st = rows3(*q, rows, hq, dh, c.type, index, "q");
    out = output(a[12], {rows, hq, dh}, c.type, index,
                 "q_out must be contiguous, as q in shape and dtype", on);
  } else if (a[12] != Py_None) {
    refuse("q_out without q");
  }
  const auto* cu = vec<int32_t>(&need_tensor(a[3], "cu_q"), int64_t(c.batch) + 1, at::kInt, index, "cu_q");
  const auto* len = vec<int32_t>(&need_tensor(a[4], "kv_len"), c.batch, at::kInt, index, "kv_len");
  const auto* pos = vec<int32_t>(maybe_tensor(a[6], "pos"), rows, at::kInt, index, "pos");
  const auto* s = vec<float>(maybe_tensor(a[7], "s"), rows, at::kFloat, index, "s");
  const auto* qn = vec<float>(maybe_tensor(a[8], "q_norm"), dh, at::kFloat, index, "q_norm");
  const auto* kn = vec<float>(maybe_tensor(a[9], "k_norm"), dh, at::kFloat, index, "k_norm");
  const double eps = PyFloat_AsDouble(a[10]), base = PyFloat_AsDouble(a[11]);
  if (PyErr_Occurred()) return nullptr;
  return finish(
      index,
      [&] {
        return tg_paged_append(&c.c, q ? q->data_ptr() : nullptr, q_st, k.data_ptr(), k_st, v.data_ptr(),
                               v_st, rows, cu, len, c.batch, hq, pos, s, qn, kn, static_cast<float>(eps),
                               static_cast<float>(base), q ? out.data_ptr() : nullptr, st);
      },
      wrap_one, q ? &out : nullptr, nullptr);
  END_HANDLE_TH_ERRORS
}

// (cache, q, cu_q, kv_len, gain, tau, max_kv, out, lse, ws, stream)
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 11)) return nullptr;
  const Cache& c = cache_of(a[0]);
  const Tensor& q = need_tensor(a[1], "q");
  if (q.dim() != 3) refuse("q must be [rows, heads, head_dim]");
  const int32_t hq = int32_of(q.size(1), "q's heads");
  const int64_t rows = q.size(0), dh = c.c.head_dim, index = c.index;
  const tg_stream st = stream_of(a[10], index);
  if (PyErr_Occurred()) return nullptr;
  const OnStream on(a[10], st, index);
  const int64_t q_st = rows3(q, rows, hq, dh, c.type, index, "q");
  Tensor out = output(a[7], {rows, hq, dh}, c.type, index,
                      "out must be contiguous, as q in shape and dtype", on);
  tg_shape shape{};
  shape.n = c.batch;
  shape.k = rows;
  shape.n_heads_q = hq;
  shape.n_heads_kv = c.c.n_heads_kv;
  shape.head_dim = c.c.head_dim;
  shape.dtype = c.c.dtype;
  const int64_t need = static_cast<int64_t>(tg_workspace_size(TG_OP_PAGED_ATTN, &shape));
  Tensor ws;
  if (a[9] != Py_None) {
    ws = need_tensor(a[9], "ws");
    const int64_t have = ws.numel() * static_cast<int64_t>(ws.element_size());
    if (have < need)
      refuse("workspace too small: " + std::to_string(have) + " < " + std::to_string(need));
    if (!ws.is_cuda() || ws.get_device() != index || !ws.is_contiguous())
      refuse("ws must be contiguous" + at_device(index));
  } else if (need > 0) {
    ws = at::empty({need}, q.options().dtype(at::kByte));
  }
  const auto* cu = vec<int32_t>(&need_tensor(a[2], "cu_q"), int64_t(c.batch) + 1, at::kInt, index, "cu_q");
  const auto* len = vec<int32_t>(&need_tensor(a[3], "kv_len"), c.batch, at::kInt, index, "kv_len");
  const auto* gain = vec<float>(maybe_tensor(a[4], "gain"), hq, at::kFloat, index, "gain");
  const auto* tau = vec<float>(maybe_tensor(a[5], "tau"), hq, at::kFloat, index, "tau");
  const auto* lse = vec<float>(maybe_tensor(a[8], "lse"), hq * rows, at::kFloat, index, "lse");
  const long long max_kv = PyLong_AsLongLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  return finish(
      index,
      [&] {
        return tg_paged_attn(&c.c, q.data_ptr(), q_st, rows, cu, len, c.batch, hq, max_kv, gain, tau, out.data_ptr(),
                             const_cast<float*>(lse), ws.defined() ? ws.data_ptr() : nullptr,
                             ws.defined() ? size_t(ws.numel()) * ws.element_size() : 0, st);
      },
      wrap_one, &out, nullptr);
  END_HANDLE_TH_ERRORS
}

// (x, xq, scale, stream)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 4)) return nullptr;
  const Tensor& x = need_tensor(a[0], "x");
  if (x.dim() != 2) refuse("x must be [rows, cols]");
  const int32_t cols = int32_of(x.size(1), "x's columns");
  const int64_t index = cuda_index(x), rows = x.size(0);
  if (x.stride(1) != 1 && rows > 0 && cols > 1) refuse("x: each row must be contiguous");
  const tg_dtype dt = dtype_of(x);
  const tg_stream st = stream_of(a[3], index);
  if (PyErr_Occurred()) return nullptr;
  const OnStream on(a[3], st, index);
  Tensor xq = output(a[1], {rows, cols}, at::kChar, index, "xq must be contiguous int8 of x's shape", on);
  Tensor scale = output(a[2], {rows}, at::kFloat, index, "scale must be contiguous fp32 [rows]", on);
  return finish(
      index,
      [&] {
        return tg_quantize_rows(x.data_ptr(), rows > 1 ? x.stride(0) : cols, rows,
                                cols, dt, static_cast<int8_t*>(xq.data_ptr()),
                                static_cast<float*>(scale.data_ptr()), st);
      },
      wrap_two, &xq, &scale);
  END_HANDLE_TH_ERRORS
}

// (xq, xs, wq, ws, residual, y, fp32 result, stream)
PyObject* linear_quantized(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 8)) return nullptr;
  const Tensor& xq = need_tensor(a[0], "xq");
  const Tensor& wq = need_tensor(a[2], "wq");
  if (xq.dim() != 2 || wq.dim() != 2) refuse("xq must be [m, k], wq [n, k]");
  const int32_t k = int32_of(xq.size(1), "k"), cols = int32_of(wq.size(0), "n");
  const int64_t index = cuda_index(xq), m = xq.size(0);
  if (wq.size(1) != k || xq.scalar_type() != at::kChar || wq.scalar_type() != at::kChar ||
      !wq.is_cuda() || wq.get_device() != index || !xq.is_contiguous() || !wq.is_contiguous())
    refuse("xq [m, k] and wq [n, k] must be contiguous int8 on one device");
  const Tensor* given = maybe_tensor(a[5], "y");
  const at::ScalarType type = given ? given->scalar_type() : a[6] == Py_True ? at::kFloat : at::kBFloat16;
  const tg_stream st = stream_of(a[7], index);
  if (PyErr_Occurred()) return nullptr;
  const OnStream on(a[7], st, index);
  Tensor y = output(a[5], {m, cols}, type, index, "y must be contiguous [m, n] on xq's device", on);
  const tg_dtype dt = dtype_of(y);
  const Tensor* res = maybe_tensor(a[4], "residual");
  if (res != nullptr && (res->sizes() != y.sizes() || res->scalar_type() != type || !res->is_cuda() ||
                         res->get_device() != index || !res->is_contiguous()))
    refuse("residual must be contiguous [m, n], as y");
  const auto* xs = vec<float>(&need_tensor(a[1], "xs"), m, at::kFloat, index, "xs");
  const auto* ws = vec<float>(&need_tensor(a[3], "ws"), cols, at::kFloat, index, "ws");
  return finish(
      index,
      [&] {
        return tg_linear_quantized(static_cast<const int8_t*>(xq.data_ptr()), xs,
                                   static_cast<const int8_t*>(wq.data_ptr()), ws,
                                   res ? res->data_ptr() : nullptr, m, cols, k, dt, y.data_ptr(), st);
      },
      wrap_one, &y, nullptr);
  END_HANDLE_TH_ERRORS
}

#define TG_METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TG_METHOD("cache", make_cache),
                         TG_METHOD("paged_append", paged_append),
                         TG_METHOD("paged_attn", paged_attn),
                         TG_METHOD("quantize_rows", quantize_rows),
                         TG_METHOD("linear_quantized", linear_quantized),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
