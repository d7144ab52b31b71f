// marshal.cpp -- the binding's short way into the attention operators (host code).
//
// A call for one token runs 3 to 6 us on the GPU; checking its ten tensors and
// converting thirty arguments in Python took 5 to 9 us more than the launch.  The
// functions here check the same things on the tensors themselves and call the
// library's entry point, whose address they are given.  They return None where
// anything is not as it should be, and the binding's own checks then say what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8bs.h"

namespace {

// A tensor argument; null where it is none of the kind asked for.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t dims) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided && t.scalar_type() == type && t.dim() == dims ? &t : nullptr;
}

// [T][H][D] whose heads are contiguous in a row.
struct Heads {
  const at::Tensor* t;
  int64_t ld, T, H, D;
};
bool heads(PyObject* o, Heads& h) {
  h.t = tensor(o, at::kBFloat16, 3);
  if (h.t == nullptr) return false;
  const auto n = h.t->sizes(), s = h.t->strides();
  h.T = n[0];
  h.H = n[1];
  h.D = n[2];
  if (s[2] != 1 || (h.H > 1 && s[1] != h.D)) return false;
  h.ld = h.T > 1 ? s[0] : std::max(s[0], h.H * h.D);
  return true;
}
// An empty tensor like it, and its row stride.
at::Tensor like(const Heads& h, int64_t& ld) {
  at::Tensor y = at::empty_like(*h.t);
  ld = h.T > 1 ? y.stride(0) : h.H * h.D;
  return y;
}

template <class T>
T* data(const at::Tensor* t) {
  return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}

bool int32s(PyObject* o, int64_t n, const at::Tensor*& t) {
  t = tensor(o, at::kInt, 1);
  return t != nullptr && t->size(0) == n && t->is_contiguous();
}

bool angles(PyObject* o, const at::Tensor*& t) {
  t = tensor(o, at::kFloat, 2);
  return t != nullptr && t->is_contiguous();
}

struct Cache {
  const at::Tensor *kc, *ks, *vc, *vs, *table, *kv_len, *q_off;
  int64_t B, Hkv, D, page, n_pages, ldt, max_pages;
};
// kc, ks, vc, vs, table, kv_len, q_off of a call with T rows.
bool cache(PyObject* const* o, int64_t T, Cache& c) {
  if (!THPVariable_Check(o[0])) return false;
  const at::ScalarType codes = THPVariable_Unpack(o[0]).scalar_type();
  if (codes != at::kByte && codes != at::kFloat8_e4m3fn) return false;
  c.kc = tensor(o[0], codes, 4);
  c.ks = tensor(o[1], at::kFloat, 2);
  c.vc = tensor(o[2], codes, 4);
  c.vs = tensor(o[3], at::kFloat, 2);
  c.table = tensor(o[4], at::kInt, 2);
  if (!c.kc || !c.ks || !c.vc || !c.vs || !c.table) return false;
  const auto n = c.kc->sizes();
  c.n_pages = n[0];
  c.Hkv = n[1];
  c.page = n[2];
  c.D = n[3];
  if (c.vc->sizes() != n || !c.kc->is_contiguous() || !c.vc->is_contiguous()) return false;
  for (const at::Tensor* s : {c.ks, c.vs})
    if (s->size(0) != c.n_pages || s->size(1) != c.Hkv || !s->is_contiguous()) return false;
  c.B = c.table->size(0);
  c.max_pages = c.table->size(1);
  if (c.table->stride(1) != 1 && c.max_pages > 1) return false;
  c.ldt = c.B > 1 ? c.table->stride(0) : std::max(c.table->stride(0), c.max_pages);
  c.q_off = nullptr;
  if (!int32s(o[5], c.B, c.kv_len)) return false;
  return o[6] == Py_None ? T == c.B : int32s(o[6], c.B + 1, c.q_off);
}

// Numbers of the call; ok turns false where one is none.
struct Numbers {
  bool ok = true;
  int64_t whole(PyObject* o) {
    if (!PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    ok = ok && over == 0;
    return x;
  }
  void* address(PyObject* o) { return reinterpret_cast<void*>(static_cast<intptr_t>(whole(o))); }
  // None: D^-1/2
  float scale(PyObject* o, int64_t D) {
    if (o == Py_None) return static_cast<float>(std::pow(static_cast<double>(D), -0.5));
    ok = ok && PyFloat_Check(o);
    return ok ? static_cast<float>(PyFloat_AS_DOUBLE(o)) : 0.0f;
  }
  // A handle, or a function that gives one: asked last, when all else is there.
  void* stream(PyObject* o) {
    if (!ok || PyLong_Check(o)) return address(o);
    PyObject* x = PyObject_CallNoArgs(o);
    if (x == nullptr) {
      PyErr_Clear();
      ok = false;
      return nullptr;
    }
    void* handle = address(x);
    Py_DECREF(x);
    return handle;
  }
};

PyObject* answer(fp8bs_status st, const at::Tensor& out) {
  if (st != FP8BS_OK) return PyLong_FromLong(st);
  return THPVariable_Wrap(out);
}

// rope(entry, x, pos, cs, rot_off, layout, inverse, stream) -> y, a status, or None
PyObject* rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads x;
  const at::Tensor *pos, *cs;
  Numbers a;
  if (n != 8 || !heads(o[1], x) || !int32s(o[2], x.T, pos) || !angles(o[3], cs)) Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_rope)>(a.address(o[0]));
  const int64_t rot_off = a.whole(o[4]);
  const int layout = static_cast<int>(a.whole(o[5])), inverse = o[6] == Py_True;
  void* stream = a.stream(o[7]);
  if (!a.ok) Py_RETURN_NONE;
  int64_t ldy;
  const at::Tensor y = like(x, ldy);
  return answer(entry(data<void>(x.t), x.ld, y.data_ptr(), ldy, data<int32_t>(pos), x.T, x.H, x.D, cs->size(1), rot_off,
                      static_cast<fp8bs_rope_layout>(layout), inverse, data<float>(cs), cs->size(0), stream),
                y);
  END_HANDLE_TH_ERRORS
}

// kv_append(entry, kc, ks, vc, vs, table, kv_len, q_off, k, v, q, cs, rot_off, layout,
// max_q, stream) -> the rotated queries, a status, or None
PyObject* kv_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads k, v, q;
  Cache c;
  const at::Tensor* cs;
  Numbers a;
  if (n != 16 || !heads(o[8], k) || !heads(o[9], v) || !heads(o[10], q) || !cache(o + 1, k.T, c) || !angles(o[11], cs))
    Py_RETURN_NONE;
  if (k.H != c.Hkv || k.D != c.D || v.T != k.T || v.H != k.H || v.D != k.D || q.T != k.T || q.D != k.D) Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_kv_append)>(a.address(o[0]));
  const int64_t rot_off = a.whole(o[12]), layout = a.whole(o[13]), max_q = a.whole(o[14]);
  void* stream = a.stream(o[15]);
  if (!a.ok) Py_RETURN_NONE;
  int64_t ldo;
  const at::Tensor y = like(q, ldo);
  return answer(entry(data<void>(q.t), q.ld, y.data_ptr(), ldo, q.H, data<void>(k.t), k.ld, data<void>(v.t), v.ld, c.Hkv,
                      c.D, data<float>(cs), cs->size(0), cs->size(1), rot_off, static_cast<fp8bs_rope_layout>(layout),
                      data<int32_t>(c.q_off), data<int32_t>(c.kv_len), c.B, k.T, max_q, data<int32_t>(c.table), c.ldt,
                      c.max_pages, c.page, data<uint8_t>(c.kc), data<float>(c.ks), data<uint8_t>(c.vc),
                      data<float>(c.vs), c.n_pages, stream),
                y);
  END_HANDLE_TH_ERRORS
}

// attn_paged(entry, kc, ks, vc, vs, table, kv_len, q_off, size entry, q, max_q, scale,
// causal, window, stream) -> out, a status, or None; on the current stream only, whose
// working memory it allocates
PyObject* attn_paged(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads q;
  Cache c;
  Numbers a;
  if (n != 15 || !heads(o[9], q) || !cache(o + 1, q.T, c) || q.D != c.D) Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_attn_paged)>(a.address(o[0]));
  const auto size = reinterpret_cast<decltype(&fp8bs_attn_paged_ws)>(a.address(o[8]));
  const int64_t max_q = a.whole(o[10]), window = a.whole(o[13]);
  const float scale = a.scale(o[11], q.D);
  const int causal = o[12] == Py_True;
  void* stream = a.stream(o[14]);
  if (!a.ok) Py_RETURN_NONE;
  int64_t ldo;
  const at::Tensor y = like(q, ldo);
  const int64_t need = size(c.B, q.T, max_q, q.H, c.Hkv, c.D, c.max_pages, c.page);
  at::Tensor ws;
  if (need > 0) ws = at::empty({need}, q.t->options().dtype(at::kByte));
  return answer(entry(data<void>(q.t), q.ld, y.data_ptr(), ldo, nullptr, 0, data<int32_t>(c.q_off), data<int32_t>(c.kv_len),
                      c.B, q.T, max_q, q.H, c.Hkv, c.D, data<int32_t>(c.table), c.ldt, c.max_pages, c.page,
                      data<uint8_t>(c.kc), data<float>(c.ks), data<uint8_t>(c.vc), data<float>(c.vs), c.n_pages, scale,
                      causal, window, need > 0 ? ws.data_ptr() : nullptr, need > 0 ? need : 0, stream),
                y);
  END_HANDLE_TH_ERRORS
}

#define FP8BS_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP8BS_METHOD(rope), FP8BS_METHOD(kv_append), FP8BS_METHOD(attn_paged), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The module looks into torch's tensors: the binding compares the version that it was
// built for before it calls anything here.
PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", FP8BS_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
