// The torch-facing calls of routing.py, dropout.py and lora.py in one step each: check the
// tensors, allocate the results on the current stream, call the C ABI. A Python body of the
// same steps takes 10 to 35 us, several times a small call's kernels.
//
// Every function returns its results, None when an argument is not what the call takes (the
// Python caller then finds out which, and says so), or the library's status when it refused.
// Memory and streams only: all arithmetic is in libmok, whose functions arrive by address
// (bind), so this module does not link against it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>

#include "mok_ops.h"

namespace {

struct Api {
  decltype(&mok_route) route;
  decltype(&mok_route_bwd) route_bwd;
  decltype(&mok_dropout) dropout;
  decltype(&mok_lora_get_sizes) lora_get_sizes;
  decltype(&mok_lora_fwd) lora_fwd;
  decltype(&mok_lora_bwd) lora_bwd;
} api;

// A dense CUDA tensor behind a Python object, or null.
const at::Tensor* dense(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided && t.is_contiguous() ? &t : nullptr;
}
// ... of a type and size, on the device of `like`
const at::Tensor* dense(PyObject* o, at::ScalarType type, int64_t numel, const at::Tensor& like) {
  const at::Tensor* t = dense(o);
  return t && t->scalar_type() == type && t->numel() == numel && t->device() == like.device()
             ? t
             : nullptr;
}
// The ABI's code of a result type, -1 for others.
int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? MOK_OUT_BF16 : t == at::kFloat ? MOK_OUT_F32 : -1;
}
at::ScalarType type_of(long code) { return code == MOK_OUT_F32 ? at::kFloat : at::kBFloat16; }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}
void* stream_of(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}
template <typename... T>
PyObject* results(T&&... tensors) {
  PyObject* out = PyTuple_New(sizeof...(tensors));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(std::move(tensors))), ...);
  return out;
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}
// The ABI struct that a ctypes object holds, copied; false (with a Python error) for others.
template <typename S>
bool read_struct(PyObject* o, S* out) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return false;
  const bool ok = b.len == (Py_ssize_t)sizeof(S);
  if (ok) std::memcpy(out, b.buf, sizeof(S));
  else PyErr_Format(PyExc_TypeError, "expected a struct of %zu bytes, got %zd", sizeof(S), b.len);
  PyBuffer_Release(&b);
  return ok;
}

// bind(route, route_bwd, dropout, lora_get_sizes, lora_fwd, lora_bwd): addresses in libmok
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 6)) return nullptr;
  api.route = reinterpret_cast<decltype(api.route)>(PyLong_AsVoidPtr(a[0]));
  api.route_bwd = reinterpret_cast<decltype(api.route_bwd)>(PyLong_AsVoidPtr(a[1]));
  api.dropout = reinterpret_cast<decltype(api.dropout)>(PyLong_AsVoidPtr(a[2]));
  api.lora_get_sizes = reinterpret_cast<decltype(api.lora_get_sizes)>(PyLong_AsVoidPtr(a[3]));
  api.lora_fwd = reinterpret_cast<decltype(api.lora_fwd)>(PyLong_AsVoidPtr(a[4]));
  api.lora_bwd = reinterpret_cast<decltype(api.lora_bwd)>(PyLong_AsVoidPtr(a[5]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// route(rule, logits, bias | None) -> (topk_idx, gates)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  mok_routing rule;
  if (!read_struct(a[0], &rule)) return nullptr;
  const at::Tensor* l = dense(a[1]);
  if (!l || l->dim() != 2 || l->size(1) != rule.E || l->size(0) > INT_MAX) Py_RETURN_NONE;
  const int code = code_of(l->scalar_type());
  const at::Tensor* b = a[2] == Py_None ? nullptr : dense(a[2], at::kFloat, rule.E, *l);
  if (code < 0 || (!b && a[2] != Py_None)) Py_RETURN_NONE;
  const int T = (int)l->size(0);
  c10::cuda::OptionalCUDAGuard guard(l->device());
  at::Tensor idx = make({T, rule.k}, at::kInt, *l), gates = make({T, rule.k}, at::kFloat, *l);
  const mok_status st = api.route(&rule, T, l->data_ptr(), (mok_out_dtype)code,
                                  b ? b->data_ptr<float>() : nullptr, idx.data_ptr<int32_t>(),
                                  gates.data_ptr<float>(), stream_of(*l));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(idx), std::move(gates));
  END_HANDLE_TH_ERRORS
}

// route_bwd(rule, logits, topk_idx, dgates, code of dlogits) -> (dlogits,)
PyObject* route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 5)) return nullptr;
  mok_routing rule;
  if (!read_struct(a[0], &rule)) return nullptr;
  const at::Tensor* l = dense(a[1]);
  if (!l || l->dim() != 2 || l->size(1) != rule.E || l->size(0) > INT_MAX) Py_RETURN_NONE;
  const int code = code_of(l->scalar_type());
  const int T = (int)l->size(0);
  const at::Tensor* idx = dense(a[2], at::kInt, (int64_t)T * rule.k, *l);
  const at::Tensor* dg = dense(a[3], at::kFloat, (int64_t)T * rule.k, *l);
  const long out_code = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  if (code < 0 || !idx || !dg) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(l->device());
  at::Tensor out = make({T, rule.E}, type_of(out_code), *l);
  const mok_status st = api.route_bwd(&rule, T, l->data_ptr(), (mok_out_dtype)code,
                                      idx->data_ptr<int32_t>(), dg->data_ptr<float>(),
                                      out.data_ptr(), (mok_out_dtype)out_code, stream_of(*l));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(out));
  END_HANDLE_TH_ERRORS
}

// dropout(x, p, seed, offset, add | None, y | None) -> (y,)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 6)) return nullptr;
  const at::Tensor* x = dense(a[0]);
  const double p = PyFloat_AsDouble(a[1]);
  const uint64_t seed = PyLong_AsUnsignedLongLongMask(a[2]);
  const uint64_t offset = PyLong_AsUnsignedLongLongMask(a[3]);
  if (PyErr_Occurred()) return nullptr;
  if (!x) Py_RETURN_NONE;
  const int code = code_of(x->scalar_type());
  const at::Tensor* add = a[4] == Py_None ? nullptr : dense(a[4], x->scalar_type(), x->numel(), *x);
  const at::Tensor* y = a[5] == Py_None ? nullptr : dense(a[5], x->scalar_type(), x->numel(), *x);
  if (code < 0 || (!add && a[4] != Py_None) || (!y && a[5] != Py_None)) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(x->device());
  at::Tensor out = y ? *y : make(x->sizes(), x->scalar_type(), *x);
  const mok_status st = api.dropout(x->data_ptr(), add ? add->data_ptr() : nullptr, out.data_ptr(),
                                    (size_t)x->numel(), (float)p, seed, offset,
                                    (mok_out_dtype)code, stream_of(*x));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(out));
  END_HANDLE_TH_ERRORS
}

// An adapted projection and its rows. weights: the tuple (W [K][N], A [n][r][K], B [n][r][N],
// scale [n], status word, (K, N, n, r)), whose tensors say at every call where they lie now; then
// x [T][K] bf16, ids [T] int32, x_ad like x or None, all on one device.
struct Adapted {
  mok_lora_dims dims;
  mok_lora_weights w;
  uint32_t* status;
  const at::Tensor *x, *ids, *x_ad;
  bool read(PyObject* weights, PyObject* px, PyObject* pids, PyObject* pad) {
    x = dense(px);
    if (!x || !PyTuple_Check(weights) || PyTuple_GET_SIZE(weights) != 6) return false;
    PyObject* sizes = PyTuple_GET_ITEM(weights, 5);
    if (!PyTuple_Check(sizes) || PyTuple_GET_SIZE(sizes) != 4) return false;
    long v[4];
    for (int i = 0; i < 4; ++i) {
      v[i] = PyLong_AsLong(PyTuple_GET_ITEM(sizes, i));
      if (v[i] < 0 || v[i] > INT_MAX) return false;
    }
    const int64_t K = v[0], N = v[1], n = v[2], r = v[3];
    auto weight = [&](int i, at::IntArrayRef shape) {
      const at::Tensor* t =
          dense(PyTuple_GET_ITEM(weights, i), at::kBFloat16, c10::multiply_integers(shape), *x);
      return t && t->sizes() == shape ? t : nullptr;
    };
    const at::Tensor *W = weight(0, {K, N}), *A = weight(1, {n, r, K}), *B = weight(2, {n, r, N}),
                     *scale = dense(PyTuple_GET_ITEM(weights, 3), at::kFloat, n, *x),
                     *word = dense(PyTuple_GET_ITEM(weights, 4), at::kInt, 1, *x);
    if (!W || !A || !B || !scale || !word) return false;
    dims = {0, (int)K, (int)N, (int)n, (int)r};
    w = {W->data_ptr(), A->data_ptr(), B->data_ptr(), scale->data_ptr<float>()};
    status = static_cast<uint32_t*>(word->data_ptr());
    if (x->scalar_type() != at::kBFloat16 || x->dim() != 2 || x->size(1) != K ||
        x->size(0) > INT_MAX)
      return false;
    dims.T = (int)x->size(0);
    ids = dense(pids, at::kInt, dims.T, *x);
    x_ad = pad == Py_None ? nullptr : dense(pad, at::kBFloat16, x->numel(), *x);
    return ids && (x_ad || pad == Py_None);
  }
};

// lora_fwd(weights, x, ids, x_ad | None, code of y) -> (y, saved)
PyObject* lora_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 5)) return nullptr;
  Adapted r;
  if (!r.read(a[0], a[1], a[2], a[3])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const long code = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  mok_lora_sizes sizes;
  mok_status st = api.lora_get_sizes(&r.dims, &sizes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  c10::cuda::OptionalCUDAGuard guard(r.x->device());
  at::Tensor y = make({r.dims.T, r.dims.N}, type_of(code), *r.x);
  at::Tensor saved = make({(int64_t)sizes.saved_bytes}, at::kByte, *r.x);
  st = api.lora_fwd(&r.dims, &r.w, r.x->data_ptr(), r.x_ad ? r.x_ad->data_ptr() : nullptr,
                    r.ids->data_ptr<int32_t>(), y.data_ptr(), (mok_out_dtype)code, saved.data_ptr(),
                    r.status, stream_of(*r.x));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(y), std::move(saved));
  END_HANDLE_TH_ERRORS
}

// lora_bwd(weights, x, ids, x_ad | None, saved, dY, code of the gradients)
//   -> (dX, dA, dB[, dXa])
PyObject* lora_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  Adapted r;
  if (!r.read(a[0], a[1], a[2], a[3])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const long code = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const mok_lora_dims& d = r.dims;
  mok_lora_sizes sizes;
  mok_status st = api.lora_get_sizes(&d, &sizes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  const at::Tensor* saved = dense(a[4], at::kByte, (int64_t)sizes.saved_bytes, *r.x);
  const at::Tensor* dY = dense(a[5], at::kBFloat16, (int64_t)d.T * d.N, *r.x);
  if (!saved || !dY) Py_RETURN_NONE;
  const at::ScalarType type = type_of(code);
  c10::cuda::OptionalCUDAGuard guard(r.x->device());
  at::Tensor dX = make({d.T, d.K}, type, *r.x), dA = make({d.n, d.r, d.K}, type, *r.x),
             dB = make({d.n, d.r, d.N}, type, *r.x), dXa;
  if (r.x_ad) dXa = make({d.T, d.K}, type, *r.x);
  const at::Tensor ws = make({(int64_t)sizes.workspace_bytes}, at::kByte, *r.x);
  st = api.lora_bwd(&d, &r.w, r.x->data_ptr(), r.x_ad ? r.x_ad->data_ptr() : nullptr,
                    r.ids->data_ptr<int32_t>(), saved->data_ptr(), dY->data_ptr(), dX.data_ptr(),
                    r.x_ad ? dXa.data_ptr() : nullptr, dA.data_ptr(), dB.data_ptr(),
                    (mok_out_dtype)code, ws.data_ptr(), r.status, stream_of(*r.x));
  if (st != MOK_OK) return PyLong_FromLong(st);
  if (r.x_ad) return results(std::move(dX), std::move(dA), std::move(dB), std::move(dXa));
  return results(std::move(dX), std::move(dA), std::move(dB));
  END_HANDLE_TH_ERRORS
}

#define MOK_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOK_CALL(bind),     MOK_CALL(route),    MOK_CALL(route_bwd),
                         MOK_CALL(dropout),  MOK_CALL(lora_fwd), MOK_CALL(lora_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mok_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mok_torch() { return PyModule_Create(&module); }
