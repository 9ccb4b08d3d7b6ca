// The torch-facing calls of routing.py, dropout.py, lora.py, norm.py, balance.py and optim.py in
// one step each: check the tensors, allocate the results on the current stream, call the C ABI. A
// Python body of the same steps takes 10 to 35 us, several times a small call's kernels.
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
#include <vector>

#include "mok_ops.h"

namespace {

struct Api {
  decltype(&mok_route) route;
  decltype(&mok_route_bwd) route_bwd;
  decltype(&mok_dropout) dropout;
  decltype(&mok_lora_get_sizes) lora_get_sizes;
  decltype(&mok_lora_fwd) lora_fwd;
  decltype(&mok_lora_bwd) lora_bwd;
  decltype(&mok_norm_get_sizes) norm_get_sizes;
  decltype(&mok_norm_fwd) norm_fwd;
  decltype(&mok_norm_bwd) norm_bwd;
  decltype(&mok_balance_get_sizes) balance_get_sizes;
  decltype(&mok_balance_fwd) balance_fwd;
  decltype(&mok_balance_bwd) balance_bwd;
  decltype(&mok_grad_norm_get_sizes) grad_norm_get_sizes;
  decltype(&mok_grad_norm) grad_norm;
  decltype(&mok_adamw) adamw;
  decltype(&mok_adamw_moments) adamw_moments;
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
// ... of the shape of `like` too
const at::Tensor* rows_like(PyObject* o, at::ScalarType type, const at::Tensor& like) {
  const at::Tensor* t = dense(o, type, like.numel(), like);
  return t && t->sizes() == like.sizes() ? t : nullptr;
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

// bind(the addresses in libmok of the functions of Api, in its order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 16)) return nullptr;
  Py_ssize_t i = 0;
  auto take = [&](auto& f) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(PyLong_AsVoidPtr(a[i++]));
  };
  take(api.route), take(api.route_bwd), take(api.dropout), take(api.lora_get_sizes);
  take(api.lora_fwd), take(api.lora_bwd), take(api.norm_get_sizes), take(api.norm_fwd);
  take(api.norm_bwd), take(api.balance_get_sizes), take(api.balance_fwd), take(api.balance_bwd);
  take(api.grad_norm_get_sizes), take(api.grad_norm), take(api.adamw), take(api.adamw_moments);
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

// A norm's parameters and rows: w [H] and b [H] or None of one type, x [T][H].
struct Normed {
  mok_norm_dims dims;
  const at::Tensor *w, *b, *x;
  bool read(PyObject* kind, PyObject* eps, PyObject* pw, PyObject* pb, PyObject* px) {
    x = dense(px);
    if (!x || x->dim() != 2 || x->size(0) > INT_MAX || x->size(1) > INT_MAX) return false;
    const int64_t H = x->size(1);
    w = dense(pw);
    if (!w || w->dim() != 1 || !dense(pw, w->scalar_type(), H, *x)) return false;
    b = pb == Py_None ? nullptr : dense(pb, w->scalar_type(), H, *x);
    if (!b && pb != Py_None) return false;
    const int xt = code_of(x->scalar_type()), wt = code_of(w->scalar_type());
    const long k = PyLong_AsLong(kind);
    const double e = PyFloat_AsDouble(eps);
    if (xt < 0 || wt < 0 || PyErr_Occurred()) return false;
    dims = {(int)x->size(0), (int)H, (int)k, (float)e, (mok_out_dtype)xt, MOK_OUT_F32,
            (mok_out_dtype)wt};
    return true;
  }
};

// norm_fwd(kind, eps, w, b | None, x, add | None, code of y) -> (y, h, stats)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  Normed r;
  if (!r.read(a[0], a[1], a[2], a[3], a[4])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const at::Tensor& x = *r.x;
  const at::Tensor* add = a[5] == Py_None ? nullptr : rows_like(a[5], x.scalar_type(), x);
  if (!add && a[5] != Py_None) Py_RETURN_NONE;
  const long code = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  r.dims.y_type = (mok_out_dtype)code;
  mok_norm_sizes sizes;
  mok_status st = api.norm_get_sizes(&r.dims, &sizes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  c10::cuda::OptionalCUDAGuard guard(x.device());
  at::Tensor y = make(x.sizes(), type_of(code), x);
  at::Tensor h = add ? make(x.sizes(), x.scalar_type(), x) : x;
  at::Tensor stats = make({x.size(0), 2}, at::kFloat, x);
  st = api.norm_fwd(&r.dims, x.data_ptr(), add ? add->data_ptr() : nullptr, r.w->data_ptr(),
                    r.b ? r.b->data_ptr() : nullptr, add ? h.data_ptr() : nullptr, y.data_ptr(),
                    stats.data_ptr<float>(), stream_of(x));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(y), std::move(h), std::move(stats));
  END_HANDLE_TH_ERRORS
}

// norm_bwd(kind, eps, w, b | None, h, dY, stats, add | None) -> (dX, dW[, dB])
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  Normed r;
  if (!r.read(a[0], a[1], a[2], a[3], a[4])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const at::Tensor& h = *r.x;
  const at::Tensor* dY = dense(a[5]);
  const int yt = dY ? code_of(dY->scalar_type()) : -1;
  if (yt < 0 || !rows_like(a[5], dY->scalar_type(), h)) Py_RETURN_NONE;
  const at::Tensor* stats = dense(a[6], at::kFloat, 2 * h.size(0), h);
  const at::Tensor* add = a[7] == Py_None ? nullptr : rows_like(a[7], h.scalar_type(), h);
  if (!stats || (!add && a[7] != Py_None)) Py_RETURN_NONE;
  r.dims.y_type = (mok_out_dtype)yt;
  mok_norm_sizes sizes;
  mok_status st = api.norm_get_sizes(&r.dims, &sizes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  c10::cuda::OptionalCUDAGuard guard(h.device());
  at::Tensor dX = make(h.sizes(), h.scalar_type(), h), dW = make({h.size(1)}, r.w->scalar_type(), h),
             dB;
  if (r.b) dB = make({h.size(1)}, r.w->scalar_type(), h);
  const at::Tensor ws = make({(int64_t)sizes.workspace_bytes}, at::kByte, h);
  st = api.norm_bwd(&r.dims, dY->data_ptr(), h.data_ptr(), r.w->data_ptr(), stats->data_ptr<float>(),
                    add ? add->data_ptr() : nullptr, dX.data_ptr(), dW.data_ptr(),
                    r.b ? dB.data_ptr() : nullptr, ws.data_ptr(), stream_of(h));
  if (st != MOK_OK) return PyLong_FromLong(st);
  if (r.b) return results(std::move(dX), std::move(dW), std::move(dB));
  return results(std::move(dX), std::move(dW));
  END_HANDLE_TH_ERRORS
}

// A router's logits [T][E] and the sequences of their rows.
struct Balanced {
  mok_balance rule;
  const at::Tensor *l, *seqs;
  int code, T, S;
  bool read(PyObject* pr, PyObject* pl, PyObject* ps) {
    if (!read_struct(pr, &rule)) return false;
    l = dense(pl);
    if (!l || l->dim() != 2 || l->size(1) != rule.E || l->size(0) > INT_MAX) return false;
    code = code_of(l->scalar_type());
    if (code < 0) return false;
    T = (int)l->size(0);
    seqs = nullptr;
    S = 1;
    if (ps != Py_None) {
      seqs = dense(ps);
      if (!seqs || seqs->dim() != 1 || seqs->size(0) < 2 || seqs->size(0) > INT_MAX ||
          !dense(ps, at::kInt, seqs->numel(), *l))
        return false;
      S = (int)seqs->size(0) - 1;
    }
    return true;
  }
  const int32_t* offsets() const { return seqs ? seqs->data_ptr<int32_t>() : nullptr; }
};

// balance_fwd(rule, logits, topk_idx, seqs | None) -> (losses, counts, saved)
PyObject* balance_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 4)) return nullptr;
  Balanced r;
  if (!r.read(a[0], a[1], a[3])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const at::Tensor* idx = dense(a[2], at::kInt, (int64_t)r.T * r.rule.k, *r.l);
  if (!idx || idx->dim() != 2 || idx->size(0) != r.T) Py_RETURN_NONE;
  size_t bytes = 0;
  mok_status st = api.balance_get_sizes(&r.rule, r.T, r.S, &bytes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  c10::cuda::OptionalCUDAGuard guard(r.l->device());
  at::Tensor losses = make({2}, at::kFloat, *r.l), counts = make({r.rule.E}, at::kInt, *r.l),
             saved = make({(int64_t)bytes}, at::kByte, *r.l);
  st = api.balance_fwd(&r.rule, r.T, r.l->data_ptr(), (mok_out_dtype)r.code,
                       idx->data_ptr<int32_t>(), r.offsets(), r.S, losses.data_ptr<float>(),
                       counts.data_ptr<int32_t>(), saved.data_ptr(), stream_of(*r.l));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(losses), std::move(counts), std::move(saved));
  END_HANDLE_TH_ERRORS
}

// balance_bwd(rule, logits, seqs | None, saved, dlosses | None, add | None, code) -> (dlogits,)
PyObject* balance_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  Balanced r;
  if (!r.read(a[0], a[1], a[2])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  size_t bytes = 0;
  mok_status st = api.balance_get_sizes(&r.rule, r.T, r.S, &bytes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  const long code = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const at::ScalarType type = type_of(code);
  const at::Tensor* saved = dense(a[3], at::kByte, (int64_t)bytes, *r.l);
  const at::Tensor* dl = a[4] == Py_None ? nullptr : dense(a[4], at::kFloat, 2, *r.l);
  const at::Tensor* add = a[5] == Py_None ? nullptr : rows_like(a[5], type, *r.l);
  if (!saved || (!dl && a[4] != Py_None) || (!add && a[5] != Py_None)) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(r.l->device());
  at::Tensor out = make(r.l->sizes(), type, *r.l);
  st = api.balance_bwd(&r.rule, r.T, r.l->data_ptr(), (mok_out_dtype)r.code, r.offsets(), r.S,
                       saved->data_ptr(), dl ? dl->data_ptr<float>() : nullptr,
                       add ? add->data_ptr() : nullptr, out.data_ptr(), (mok_out_dtype)code,
                       stream_of(*r.l));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(out));
  END_HANDLE_TH_ERRORS
}

// The items of a list or tuple, without a reference of their own.
bool items(PyObject* o, PyObject*** at, Py_ssize_t* n) {
  if (!PyList_Check(o) && !PyTuple_Check(o)) return false;
  *at = PySequence_Fast_ITEMS(o);
  *n = PySequence_Fast_GET_SIZE(o);
  return *n <= INT_MAX;
}

// grad_norm([tensor | None, ...], max_norm, scale) -> (norm, coef)
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  PyObject** g;
  Py_ssize_t tensors;
  if (!items(a[0], &g, &tensors)) Py_RETURN_NONE;
  const double max_norm = PyFloat_AsDouble(a[1]), scale = PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* like = nullptr;
  std::vector<mok_grad> grads((size_t)tensors);
  for (Py_ssize_t i = 0; i < tensors; ++i) {
    if (g[i] == Py_None) continue;
    const at::Tensor* t = dense(g[i]);
    const int code = t ? code_of(t->scalar_type()) : -1;
    if (code < 0 || (like && t->device() != like->device())) Py_RETURN_NONE;
    like = t;
    grads[i] = {t->data_ptr(), (size_t)t->numel(), (mok_out_dtype)code};
  }
  if (!like) Py_RETURN_NONE;
  size_t bytes = 0;
  mok_status st = api.grad_norm_get_sizes(&bytes);
  if (st != MOK_OK) return PyLong_FromLong(st);
  c10::cuda::OptionalCUDAGuard guard(like->device());
  at::Tensor norm = make({1}, at::kFloat, *like), coef = make({1}, at::kFloat, *like);
  const at::Tensor ws = make({(int64_t)bytes}, at::kByte, *like);
  st = api.grad_norm((int)tensors, grads.data(), (float)max_norm, (float)scale,
                     norm.data_ptr<float>(), coef.data_ptr<float>(), ws.data_ptr(),
                     stream_of(*like));
  if (st != MOK_OK) return PyLong_FromLong(st);
  return results(std::move(norm), std::move(coef));
  END_HANDLE_TH_ERRORS
}

// Whether two tensors of as many elements hold them in one order: one shape, or a flat view of it.
bool same_order(const at::Tensor& a, const at::Tensor& b) {
  return a.dim() <= 1 || b.dim() <= 1 || a.sizes() == b.sizes();
}

// adamw(rule, params, what, (master | None, m, v, scales | None), elements, grads, lr, t, coef | None,
//       seed) -> ()
// params: a tuple of tensors; what: an array of mok_adamw_tensor with their sizes, types and decays,
// which the state was made for; grads: a list or tuple of a tensor or None for each; lr and t:
// numbers, or tensors of one fp32 and one int32 value.
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  mok_adamw_rule rule;
  if (!read_struct(a[0], &rule)) return nullptr;
  PyObject **p, **st, **g;
  Py_ssize_t np, ns, ng;
  if (!items(a[1], &p, &np) || !items(a[3], &st, &ns) || !items(a[5], &g, &ng) || np != ng || ns != 4)
    Py_RETURN_NONE;
  std::vector<mok_adamw_tensor> tensors((size_t)np);
  Py_buffer b;
  if (PyObject_GetBuffer(a[2], &b, PyBUF_SIMPLE) != 0) return nullptr;
  const bool fits = b.len == np * (Py_ssize_t)sizeof(mok_adamw_tensor);
  if (fits) std::memcpy(tensors.data(), b.buf, (size_t)b.len);
  PyBuffer_Release(&b);
  if (!fits) Py_RETURN_NONE;
  const at::Tensor* m = dense(st[1]);
  if (!m) Py_RETURN_NONE;
  const int64_t elements = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  const bool small = rule.bits == 8;
  const at::ScalarType kind = small ? at::kByte : at::kFloat;
  const at::Tensor* master = st[0] == Py_None ? nullptr : dense(st[0], at::kFloat, elements, *m);
  const at::Tensor* v = dense(st[2], kind, elements, *m);
  const at::Tensor* scales = small ? dense(st[3], at::kByte, elements / 128, *m) : nullptr;
  if (!dense(st[1], kind, elements, *m) || !v || (!master && st[0] != Py_None) || (small && !scales))
    Py_RETURN_NONE;
  for (Py_ssize_t i = 0; i < np; ++i) {
    mok_adamw_tensor& x = tensors[i];
    const at::Tensor* t = dense(p[i], type_of(x.p_type), (int64_t)x.n, *m);
    if (!t) Py_RETURN_NONE;
    x.p = t->data_ptr();
    x.g = nullptr;
    x.g_type = MOK_OUT_F32;
    if (g[i] == Py_None) continue;
    const at::Tensor* d = dense(g[i]);
    const int code = d ? code_of(d->scalar_type()) : -1;
    if (code < 0 || d->numel() != (int64_t)x.n || d->device() != m->device() || !same_order(*d, *t)) Py_RETURN_NONE;
    x.g = d->data_ptr();
    x.g_type = (mok_out_dtype)code;
  }
  double lr = 0.;
  long t = 1;
  const at::Tensor *lr_dev = nullptr, *t_dev = nullptr;
  if (THPVariable_Check(a[6])) {
    if (!(lr_dev = dense(a[6], at::kFloat, 1, *m))) Py_RETURN_NONE;
  } else {
    lr = PyFloat_AsDouble(a[6]);
  }
  if (THPVariable_Check(a[7])) {
    if (!(t_dev = dense(a[7], at::kInt, 1, *m))) Py_RETURN_NONE;
  } else {
    t = PyLong_AsLong(a[7]);
  }
  if (PyErr_Occurred()) return nullptr;
  if (t > INT_MAX || t < 1) return PyLong_FromLong(MOK_ERR_INVALID_ARG);
  const at::Tensor* coef = a[8] == Py_None ? nullptr : dense(a[8], at::kFloat, 1, *m);
  if (!coef && a[8] != Py_None) Py_RETURN_NONE;
  const uint64_t seed = PyLong_AsUnsignedLongLongMask(a[9]);
  if (PyErr_Occurred()) return nullptr;
  c10::cuda::OptionalCUDAGuard guard(m->device());
  const mok_adamw_state state = {master ? master->data_ptr<float>() : nullptr, m->data_ptr(),
                                 v->data_ptr(),
                                 scales ? scales->data_ptr<uint8_t>() : nullptr};
  const mok_status s = api.adamw(&rule, (int)np, tensors.data(), &state, lr,
                                 lr_dev ? lr_dev->data_ptr<float>() : nullptr, (int)t,
                                 t_dev ? t_dev->data_ptr<int32_t>() : nullptr,
                                 coef ? coef->data_ptr<float>() : nullptr, seed, stream_of(*m));
  if (s != MOK_OK) return PyLong_FromLong(s);
  return PyTuple_New(0);
  END_HANDLE_TH_ERRORS
}

// adamw_moments(m, v, scales) -> (m, v) in bf16
PyObject* adamw_moments(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  const at::Tensor* m = dense(a[0]);
  if (!m || m->scalar_type() != at::kByte) Py_RETURN_NONE;
  const at::Tensor* v = dense(a[1], at::kByte, m->numel(), *m);
  const at::Tensor* scales = dense(a[2], at::kByte, m->numel() / 128, *m);
  if (!v || !scales) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(m->device());
  at::Tensor mo = make({m->numel()}, at::kBFloat16, *m), vo = make({m->numel()}, at::kBFloat16, *m);
  const mok_adamw_state state = {nullptr, m->data_ptr(), v->data_ptr(), scales->data_ptr<uint8_t>()};
  const mok_status s = api.adamw_moments((size_t)m->numel(), &state, mo.data_ptr(), vo.data_ptr(),
                                         stream_of(*m));
  if (s != MOK_OK) return PyLong_FromLong(s);
  return results(std::move(mo), std::move(vo));
  END_HANDLE_TH_ERRORS
}

#define MOK_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOK_CALL(bind),     MOK_CALL(route),    MOK_CALL(route_bwd),
                         MOK_CALL(dropout),  MOK_CALL(lora_fwd), MOK_CALL(lora_bwd),
                         MOK_CALL(norm_fwd), MOK_CALL(norm_bwd), MOK_CALL(balance_fwd),
                         MOK_CALL(balance_bwd), MOK_CALL(grad_norm), MOK_CALL(adamw),
                         MOK_CALL(adamw_moments),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mok_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mok_torch() { return PyModule_Create(&module); }
