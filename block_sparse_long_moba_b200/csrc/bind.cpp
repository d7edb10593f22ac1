// Argument marshalling for the latency-bound calls of moba.py (norm + rotary, paged cache): the
// conditions under which a call is plain - tensors of the right type, shape and device, on the
// current stream - are checked here in well under a microsecond, outputs and workspace that were
// not given are allocated, and the C entry point of libmoba.so is called. Where a condition does
// not hold the function returns None, and moba.py's own checks say what is wrong. No computation
// happens here; a decode step's calls take a few microseconds on the GPU, and checking ten tensors
// from Python costs more than that.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moba.h"

namespace {

struct Entry {
  decltype(&moba_qk_norm_rope) norm;
  decltype(&moba_qk_norm_rope_bwd) norm_bwd;
  decltype(&moba_qk_norm_rope_bwd_workspace_bytes) norm_bwd_bytes;
  decltype(&moba_cache_append) append;
  decltype(&moba_cache_read) read;
  decltype(&moba_paged_attn_fwd) attn;
  decltype(&moba_paged_decode_fwd) decode;
};
Entry fn{};

constexpr auto kBf16 = at::kBFloat16;

// The tensor behind an argument, or null.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}
bool is(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev &&
         t->sizes() == shape && t->is_contiguous();
}
// bf16 [T, heads, d] whose heads are packed; the token stride in elements.
bool rows(const at::Tensor* t, int dev, long long* ld) {
  if (!t || t->scalar_type() != kBf16 || !t->is_cuda() || t->get_device() != dev || t->dim() != 3)
    return false;
  const auto s = t->sizes(), st = t->strides();
  if ((s[2] > 1 && st[2] != 1) || (s[1] > 1 && st[1] != s[2])) return false;
  *ld = s[0] > 1 ? st[0] : s[1] * s[2];
  return true;
}
// The output given, or a new one; false when what was given does not fit.
bool output(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int dev, at::Tensor* t) {
  if (o == Py_None) {
    *t = at::empty(shape, at::TensorOptions(type).device(at::kCUDA, dev));
    return true;
  }
  const at::Tensor* g = tensor(o);
  if (!is(g, type, shape, dev)) return false;
  *t = *g;
  return true;
}
at::Tensor workspace(size_t bytes, int dev) {
  return at::empty({static_cast<int64_t>(bytes < 256 ? 256 : bytes)},
                   at::TensorOptions(at::kByte).device(at::kCUDA, dev));
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const auto& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// init(addresses...): the entry points of the loaded library.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "init takes seven addresses");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  fn.norm = reinterpret_cast<decltype(fn.norm)>(p[0]);
  fn.norm_bwd = reinterpret_cast<decltype(fn.norm_bwd)>(p[1]);
  fn.norm_bwd_bytes = reinterpret_cast<decltype(fn.norm_bwd_bytes)>(p[2]);
  fn.append = reinterpret_cast<decltype(fn.append)>(p[3]);
  fn.read = reinterpret_cast<decltype(fn.read)>(p[4]);
  fn.attn = reinterpret_cast<decltype(fn.attn)>(p[5]);
  fn.decode = reinterpret_cast<decltype(fn.decode)>(p[6]);
  Py_RETURN_NONE;
}

struct Norm {
  const at::Tensor *q, *k, *wq, *wk, *rope, *pos;
  long long q_ld, k_ld;
  int dev, T, Hq, Hkv, d;
};
bool norm_args(PyObject* const* a, Norm* N) {
  if (!fn.norm) return false;
  N->q = tensor(a[0]); N->k = tensor(a[1]); N->wq = tensor(a[2]);
  N->wk = tensor(a[3]); N->rope = tensor(a[4]); N->pos = tensor(a[5]);
  if (!N->q || !N->q->is_cuda()) return false;
  N->dev = c10::cuda::current_device();
  if (!rows(N->q, N->dev, &N->q_ld) || !rows(N->k, N->dev, &N->k_ld)) return false;
  const int64_t T = N->q->size(0), d = N->q->size(2);
  if (N->k->size(0) != T || N->k->size(2) != d || T > INT_MAX || N->q->size(1) > INT_MAX ||
      N->k->size(1) > INT_MAX || d > INT_MAX)
    return false;
  N->T = static_cast<int>(T);
  N->Hq = static_cast<int>(N->q->size(1));
  N->Hkv = static_cast<int>(N->k->size(1));
  N->d = static_cast<int>(d);
  return is(N->wq, at::kFloat, {d}, N->dev) && is(N->wk, at::kFloat, {d}, N->dev) && N->rope &&
         N->rope->dim() == 2 && N->rope->size(0) <= INT_MAX && N->rope->size(1) <= INT_MAX &&
         is(N->rope, at::kFloat, N->rope->sizes(), N->dev) && is(N->pos, at::kInt, {T}, N->dev);
}

// norm_rope(q, k, q_weight, k_weight, rope, positions, eps, interleaved, q_out, k_out)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Norm N;
  if (n != 10 || !norm_args(a, &N)) Py_RETURN_NONE;
  const double eps = PyFloat_AsDouble(a[6]);
  const int adj = PyObject_IsTrue(a[7]);
  if (PyErr_Occurred()) return nullptr;
  at::Tensor qo, ko;
  if (!output(a[8], kBf16, {N.T, N.Hq, N.d}, N.dev, &qo) ||
      !output(a[9], kBf16, {N.T, N.Hkv, N.d}, N.dev, &ko))
    Py_RETURN_NONE;
  const int st = fn.norm(N.q->data_ptr(), N.q_ld, N.k->data_ptr(), N.k_ld,
                         N.wq->data_ptr<float>(), N.wk->data_ptr<float>(),
                         N.rope->data_ptr<float>(), static_cast<int>(N.rope->size(0)),
                         static_cast<int>(N.rope->size(1)), N.pos->data_ptr<int>(), N.T, N.Hq,
                         N.Hkv, N.d, static_cast<float>(eps), adj, qo.data_ptr(), ko.data_ptr(),
                         stream_of(N.dev));
  return st ? PyLong_FromLong(st) : pack({qo, ko});
  END_HANDLE_TH_ERRORS
}

// norm_rope_bwd(q, k, q_weight, k_weight, rope, positions, d_q_out, d_k_out, eps, interleaved)
PyObject* norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Norm N;
  if (n != 10 || !norm_args(a, &N)) Py_RETURN_NONE;
  const at::Tensor *dyq = tensor(a[6]), *dyk = tensor(a[7]);
  const double eps = PyFloat_AsDouble(a[8]);
  const int adj = PyObject_IsTrue(a[9]);
  if (PyErr_Occurred()) return nullptr;
  if (!is(dyq, kBf16, {N.T, N.Hq, N.d}, N.dev) || !is(dyk, kBf16, {N.T, N.Hkv, N.d}, N.dev))
    Py_RETURN_NONE;
  at::Tensor dq = at::empty_like(*dyq), dk = at::empty_like(*dyk);
  at::Tensor dwq = at::empty_like(*N.wq), dwk = at::empty_like(*N.wk);
  at::Tensor ws = workspace(fn.norm_bwd_bytes(N.Hq, N.Hkv, N.d), N.dev);
  const int st = fn.norm_bwd(
      N.q->data_ptr(), N.q_ld, N.k->data_ptr(), N.k_ld, N.wq->data_ptr<float>(),
      N.wk->data_ptr<float>(), N.rope->data_ptr<float>(), static_cast<int>(N.rope->size(0)),
      static_cast<int>(N.rope->size(1)), N.pos->data_ptr<int>(), dyq->data_ptr(), dyk->data_ptr(),
      N.T, N.Hq, N.Hkv, N.d, static_cast<float>(eps), adj, dq.data_ptr(), dk.data_ptr(),
      dwq.data_ptr<float>(), dwk.data_ptr<float>(), ws.data_ptr(),
      static_cast<size_t>(ws.numel()), stream_of(N.dev));
  return st ? PyLong_FromLong(st) : pack({dq, dk, dwq, dwk});
  END_HANDLE_TH_ERRORS
}

// The cache of a call: (address of the moba_paged_cache, device index).
struct Cache {
  const moba_paged_cache* c;
  int dev;
};
bool cache_args(PyObject* const* a, Cache* C) {
  C->c = static_cast<const moba_paged_cache*>(PyLong_AsVoidPtr(a[0]));
  C->dev = static_cast<int>(PyLong_AsLong(a[1]));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return fn.norm && C->c && C->dev >= 0 && C->dev == c10::cuda::current_device();
}

// append(cache, device, k, v, cu_seqlens_q): the status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache C;
  if (n != 5 || !cache_args(a, &C)) Py_RETURN_NONE;
  const at::Tensor *k = tensor(a[2]), *v = tensor(a[3]), *cu = tensor(a[4]);
  long long k_ld, v_ld;
  if (!rows(k, C.dev, &k_ld) || !rows(v, C.dev, &v_ld) || k->sizes() != v->sizes() ||
      k->size(1) != C.c->Hkv || k->size(2) != C.c->d || k->size(0) > INT_MAX ||
      !is(cu, at::kInt, {C.c->nseq + 1}, C.dev))
    Py_RETURN_NONE;
  return PyLong_FromLong(fn.append(C.c, k->data_ptr(), k_ld, v->data_ptr(), v_ld,
                                   cu->data_ptr<int>(), static_cast<int>(k->size(0)),
                                   stream_of(C.dev)));
  END_HANDLE_TH_ERRORS
}

// read(cache, device, cu_seqlens, T, k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache C;
  if (n != 6 || !cache_args(a, &C)) Py_RETURN_NONE;
  const at::Tensor* cu = tensor(a[2]);
  const long T = PyLong_AsLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  if (T < 0 || T > INT_MAX || !is(cu, at::kInt, {C.c->nseq + 1}, C.dev)) Py_RETURN_NONE;
  at::Tensor k, v;
  if (!output(a[4], kBf16, {T, C.c->Hkv, C.c->d}, C.dev, &k) ||
      !output(a[5], kBf16, {T, C.c->Hkv, C.c->d}, C.dev, &v))
    Py_RETURN_NONE;
  const int st = fn.read(C.c, cu->data_ptr<int>(), static_cast<int>(T), k.data_ptr(),
                         v.data_ptr(), stream_of(C.dev));
  return st ? PyLong_FromLong(st) : pack({k, v});
  END_HANDLE_TH_ERRORS
}

// paged(cache, device, q, rows_per_seq, topk, scale, block_idx_out, o, lse, workspace,
//       workspace_bytes): topk 0 for full attention
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache C;
  if (n != 11 || !cache_args(a, &C)) Py_RETURN_NONE;
  const at::Tensor* q = tensor(a[2]);
  const long nrow = PyLong_AsLong(a[3]), topk = PyLong_AsLong(a[4]);
  const double scale = PyFloat_AsDouble(a[5]);
  const size_t bytes = PyLong_AsSize_t(a[10]);
  if (PyErr_Occurred()) return nullptr;
  if (!q || q->dim() != 3 || nrow < 1 || nrow > INT_MAX || topk < 0 || topk > INT_MAX)
    Py_RETURN_NONE;
  const int64_t R = static_cast<int64_t>(C.c->nseq) * nrow, hq = q->size(1);
  if (hq > INT_MAX || !is(q, kBf16, {R, hq, C.c->d}, C.dev)) Py_RETURN_NONE;
  int* idx = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor* t = tensor(a[6]);
    if (!is(t, at::kInt, {hq, R, topk}, C.dev)) Py_RETURN_NONE;
    idx = t->data_ptr<int>();
  }
  at::Tensor o, lse, ws;
  if (!output(a[7], kBf16, {R, hq, C.c->d}, C.dev, &o) ||
      !output(a[8], at::kFloat, {hq, R}, C.dev, &lse))
    Py_RETURN_NONE;
  if (a[9] == Py_None) {
    ws = workspace(bytes, C.dev);
  } else {
    const at::Tensor* t = tensor(a[9]);
    if (!t || !is(t, at::kByte, t->sizes(), C.dev)) Py_RETURN_NONE;
    ws = *t;
  }
  const int st =
      topk ? fn.decode(C.c, q->data_ptr(), static_cast<int>(hq), static_cast<int>(nrow),
                       static_cast<int>(topk), static_cast<float>(scale), idx, o.data_ptr(),
                       lse.data_ptr<float>(), ws.data_ptr(), static_cast<size_t>(ws.numel()),
                       stream_of(C.dev))
           : fn.attn(C.c, q->data_ptr(), static_cast<int>(hq), static_cast<int>(nrow),
                     static_cast<float>(scale), o.data_ptr(), lse.data_ptr<float>(),
                     ws.data_ptr(), static_cast<size_t>(ws.numel()), stream_of(C.dev));
  return st ? PyLong_FromLong(st) : pack({o, lse});
  END_HANDLE_TH_ERRORS
}

#define MOBA_METHOD(name, doc) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, doc}
PyMethodDef methods[] = {
    MOBA_METHOD(init, "entry points of the loaded library"),
    MOBA_METHOD(norm_rope, "moba_qk_norm_rope: (q_out, k_out), a status, or None"),
    MOBA_METHOD(norm_rope_bwd, "moba_qk_norm_rope_bwd: the gradients, a status, or None"),
    MOBA_METHOD(append, "moba_cache_append: a status, or None"),
    MOBA_METHOD(read, "moba_cache_read: (k, v), a status, or None"),
    MOBA_METHOD(paged, "moba_paged_attn_fwd / _decode_fwd: (o, lse), a status, or None"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", MOBA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
