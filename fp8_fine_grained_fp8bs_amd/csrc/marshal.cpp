// marshal.cpp -- the binding's short way into the attention operators and those
// around the experts' products (host code).
//
// A call for one token runs 3 to 6 us on the GPU; checking its ten tensors and
// converting thirty arguments in Python took 5 to 9 us more than the launch.  The
// functions here check the same things on the tensors themselves and call the
// library's entry point, whose address they are given.  They return None where
// anything is not as it should be, and the binding's own checks then say what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
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
  bool flag(PyObject* o) {
    ok = ok && PyBool_Check(o);
    return o == Py_True;
  }
  float real(PyObject* o) {
    ok = ok && PyFloat_Check(o);
    return ok ? static_cast<float>(PyFloat_AS_DOUBLE(o)) : 0.0f;
  }
  // A handle, a function that gives one (asked last, when all else is there), or None:
  // the current device's current stream.
  void* stream(PyObject* o) {
    if (o == Py_None) return c10::hip::getCurrentHIPStream().stream();
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

// [rows][cols] with contiguous rows.
struct Matrix {
  const at::Tensor* t = nullptr;
  int64_t ld = 0, rows = 0, cols = 0;
};
bool matrix(PyObject* o, at::ScalarType type, Matrix& m) {
  m.t = tensor(o, type, 2);
  if (m.t == nullptr || m.t->stride(1) != 1) return false;
  m.rows = m.t->size(0);
  m.cols = m.t->size(1);
  m.ld = m.rows > 1 ? m.t->stride(0) : m.cols;   // a single row's stride does not matter
  return true;
}
bool matrix(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols, Matrix& m) {
  return matrix(o, type, m) && m.rows == rows && m.cols == cols;
}
// The same, or None.
bool optional(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols, Matrix& m) {
  return o == Py_None || matrix(o, type, rows, cols, m);
}
// In BF16 or FP32; f32 says which.
bool values(PyObject* o, Matrix& m, bool& f32) {
  f32 = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kFloat;
  return matrix(o, f32 ? at::kFloat : at::kBFloat16, m);
}
bool codes(PyObject* o, Matrix& m) {
  const bool bytes = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kByte;
  return matrix(o, bytes ? at::kByte : at::kFloat8_e4m3fn, m);
}
bool vector(PyObject* o, at::ScalarType type, int64_t n, const at::Tensor*& t) {
  t = tensor(o, type, 1);
  return t != nullptr && t->size(0) == n && t->is_contiguous();
}
bool gamma_of(PyObject* o, int64_t C, const at::Tensor*& t, fp8bs_out_dtype& type) {
  const bool f32 = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kFloat;
  type = f32 ? FP8BS_OUT_F32 : FP8BS_OUT_BF16;
  return vector(o, f32 ? at::kFloat : at::kBFloat16, C, t);
}
fp8bs_out_dtype type_of(bool f32) { return f32 ? FP8BS_OUT_F32 : FP8BS_OUT_BF16; }

// Whether all of them (null: not given) are on the current device, on which the kernels run.
bool here(std::initializer_list<const at::Tensor*> tensors) {
  const auto device = c10::hip::current_device();
  for (const at::Tensor* t : tensors)
    if (t != nullptr && t->device().index() != device) return false;
  return true;
}

// A new [rows][cols] on x's device where wanted, and its pointer.
struct Fresh {
  at::Tensor t;
  Fresh(const at::Tensor* x, bool wanted, at::ScalarType type, at::IntArrayRef size) {
    if (wanted) t = at::Tensor(at::detail::empty_cuda(size, type, x->device(), std::nullopt));
  }
  template <class T>
  T* data() const {
    return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
  }
};
// Row outputs: codes with scales and BF16 rows, given as tensors or made.
struct Rows {
  Fresh q, s, y;
  PyObject* given[3] = {nullptr, nullptr, nullptr};
  Matrix mq, ms, my;
  int64_t M = 0, cols;
  Rows(const at::Tensor* x, bool codes, bool bf16, int64_t rows, int64_t cols)
      : q(x, codes, at::kByte, {rows, cols}), s(x, codes, at::kFloat, {rows, cols / 128}),
        y(x, bf16, at::kBFloat16, {rows, cols}), M(rows), cols(cols) {}
  // (q, s, y) of a caller: false where they do not fit
  bool take(PyObject* out) {
    if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != 3) return false;
    for (int i = 0; i < 3; ++i) given[i] = PyTuple_GET_ITEM(out, i);
    M = -1;
    if ((given[0] == Py_None) != (given[1] == Py_None)) return false;
    if (given[0] != Py_None) {
      if (!::codes(given[0], mq) || mq.cols != cols) return false;
      M = mq.rows;
      if (!matrix(given[1], at::kFloat, ms) || ms.rows != M || ms.cols < cols / 128) return false;
    }
    if (given[2] != Py_None) {
      if (!matrix(given[2], at::kBFloat16, my) || my.cols != cols || (M >= 0 && my.rows != M)) return false;
      M = my.rows;
    }
    return M >= 0;
  }
  uint8_t* pq() const { return mq.t != nullptr ? static_cast<uint8_t*>(mq.t->data_ptr()) : q.data<uint8_t>(); }
  float* ps() const { return ms.t != nullptr ? data<float>(ms.t) : s.data<float>(); }
  void* py() const { return my.t != nullptr ? my.t->data_ptr() : y.data<void>(); }
  int64_t ldq() const { return mq.t != nullptr ? mq.ld : cols; }
  int64_t lds() const { return ms.t != nullptr ? ms.ld : cols / 128; }
  int64_t ldy() const { return my.t != nullptr ? my.ld : cols; }
};

// The outputs as a tuple (a caller's own where given, None for those not made), or the status.
struct Output {
  PyObject* given;
  const at::Tensor* made;
  Output(const Fresh& f) : given(nullptr), made(&f.t) {}
  Output(PyObject* given, const Fresh& f) : given(given), made(&f.t) {}
};
PyObject* answers(fp8bs_status st, std::initializer_list<Output> outputs) {
  if (st != FP8BS_OK) return PyLong_FromLong(st);
  PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(outputs.size()));
  if (all == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Output& o : outputs) {
    PyObject* x = o.given != nullptr ? o.given : o.made->defined() ? nullptr : Py_None;
    if (x != nullptr) Py_INCREF(x);
    else x = THPVariable_Wrap(*o.made);
    if (x == nullptr) {
      Py_DECREF(all);
      return nullptr;
    }
    PyTuple_SET_ITEM(all, i++, x);
  }
  return all;
}

// rmsnorm_quant_1x128(entry, x, gamma, residual, eps, codes, with_y, with_rstd, stream)
// -> (q, s, h, y, rstd), a status, or None
PyObject* rmsnorm_quant_1x128(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Matrix x, r;
  const at::Tensor* gamma;
  fp8bs_out_dtype gt;
  Numbers a;
  if (n != 9 || !matrix(o[1], at::kBFloat16, x) || !optional(o[3], at::kBFloat16, x.rows, x.cols, r) ||
      !gamma_of(o[2], x.cols, gamma, gt))
    Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_rmsnorm_quant_1x128)>(a.address(o[0]));
  const float eps = a.real(o[4]);
  const bool with_q = a.flag(o[5]), with_y = a.flag(o[6]), with_rstd = a.flag(o[7]);
  void* stream = a.stream(o[8]);
  if (!a.ok || (!with_q && !with_y) || !here({x.t, r.t, gamma})) Py_RETURN_NONE;
  const Rows out(x.t, with_q, with_y, x.rows, x.cols);
  const Fresh h(x.t, r.t != nullptr, at::kBFloat16, {x.rows, x.cols}), rstd(x.t, with_rstd, at::kFloat, {x.rows});
  return answers(entry(data<void>(x.t), x.ld, data<void>(r.t), r.ld, data<void>(gamma), gt, eps, x.rows, x.cols,
                       h.data<void>(), x.cols, out.pq(), out.ldq(), out.ps(), out.lds(), out.py(), out.ldy(),
                       rstd.data<float>(), stream),
                 {out.q, out.s, h, out.y, rstd});
  END_HANDLE_TH_ERRORS
}

// rmsnorm_bwd(entry, size entry, dn, h, gamma, rstd, dres, with_dgamma, stream)
// -> (dx, dgamma), a status, or None
PyObject* rmsnorm_bwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Matrix dn, h, dres;
  const at::Tensor *gamma, *rstd;
  fp8bs_out_dtype gt;
  Numbers a;
  if (n != 9 || !matrix(o[3], at::kBFloat16, h) || !matrix(o[2], at::kBFloat16, h.rows, h.cols, dn) ||
      !gamma_of(o[4], h.cols, gamma, gt) || !vector(o[5], at::kFloat, h.rows, rstd) ||
      !optional(o[6], at::kBFloat16, h.rows, h.cols, dres))
    Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_rmsnorm_bwd)>(a.address(o[0]));
  const auto size = reinterpret_cast<decltype(&fp8bs_rmsnorm_bwd_ws)>(a.address(o[1]));
  const bool with = a.flag(o[7]);
  void* stream = a.stream(o[8]);
  if (!a.ok || !here({dn.t, h.t, dres.t, gamma, rstd})) Py_RETURN_NONE;
  const int64_t need = with ? std::max<int64_t>(size(h.rows, h.cols), 0) : 0;
  const Fresh dx(h.t, true, at::kBFloat16, {h.rows, h.cols}), dgamma(h.t, with, at::kFloat, {h.cols}),
      ws(h.t, need > 0, at::kByte, {need});
  return answers(entry(data<void>(dn.t), dn.ld, data<void>(dres.t), dres.ld, data<void>(h.t), h.ld, data<void>(gamma), gt,
                       data<float>(rstd), h.rows, h.cols, dx.data<void>(), h.cols, dgamma.data<float>(), ws.data<void>(),
                       need, stream),
                 {dx, dgamma});
  END_HANDLE_TH_ERRORS
}

// moe_dispatch(entry, size entry, x, s_in, ids, E, first, rows, codes, with_y, out, stream)
// -> (q, s, y, offsets, slot), a status, or None; rows None: all
PyObject* moe_dispatch(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Matrix x, s_in, ids;
  Numbers a;
  if (n != 12) Py_RETURN_NONE;
  const bool bf16 = o[3] == Py_None;
  if (bf16 ? !matrix(o[2], at::kBFloat16, x)
           : !codes(o[2], x) || !matrix(o[3], at::kFloat, s_in) || s_in.rows != x.rows || s_in.cols < x.cols / 128)
    Py_RETURN_NONE;
  const bool wide = THPVariable_Check(o[4]) && THPVariable_Unpack(o[4]).scalar_type() == at::kLong;
  if (!matrix(o[4], wide ? at::kLong : at::kInt, ids) || ids.rows != x.rows) Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_moe_dispatch)>(a.address(o[0]));
  const auto size = reinterpret_cast<decltype(&fp8bs_moe_sort_ws)>(a.address(o[1]));
  const int64_t E = a.whole(o[5]), first = a.whole(o[6]), k = ids.cols;
  const int64_t rows = o[7] == Py_None ? x.rows * k : a.whole(o[7]);
  const bool with_q = a.flag(o[8]), with_y = a.flag(o[9]), made = o[10] == Py_None;
  void* stream = a.stream(o[11]);
  if (!a.ok || E <= 0 || E > (1 << 20) || rows < 0) Py_RETURN_NONE;
  Rows out(x.t, made && with_q, made && with_y, rows, x.cols);
  if (!made && !out.take(o[10])) Py_RETURN_NONE;
  if (!here({x.t, s_in.t, ids.t, out.mq.t, out.ms.t, out.my.t})) Py_RETURN_NONE;
  const int64_t need = std::max<int64_t>(size(x.rows, k, E), 0);
  const Fresh offsets(x.t, true, at::kInt, {E + 1}), slot(x.t, true, at::kInt, {x.rows, k}),
      ws(x.t, need > 0, at::kByte, {need});
  return answers(entry(bf16 ? FP8BS_SRC_BF16 : FP8BS_SRC_FP8_1x128, data<void>(x.t), x.ld, data<float>(s_in.t), s_in.ld,
                       x.rows, x.cols, data<void>(ids.t), wide ? FP8BS_INDEX_I64 : FP8BS_INDEX_I32, ids.ld, k, first, E,
                       offsets.data<int32_t>(), slot.data<int32_t>(), out.pq(), out.ldq(), out.ps(), out.lds(), out.py(),
                       out.ldy(), out.M, ws.data<void>(), need, stream),
                 {{out.given[0], out.q}, {out.given[1], out.s}, {out.given[2], out.y}, offsets, slot});
  END_HANDLE_TH_ERRORS
}

bool slots(PyObject* o, const at::Tensor*& t) {
  t = tensor(o, at::kInt, 2);
  return t != nullptr && t->is_contiguous();
}

// moe_combine(entry, y, slot, w, add, stream) -> out, a status, or None
PyObject* moe_combine(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Matrix y, w, add;
  bool f32;
  const at::Tensor* slot;
  Numbers a;
  if (n != 6 || !values(o[1], y, f32) || !slots(o[2], slot)) Py_RETURN_NONE;
  const int64_t T = slot->size(0), k = slot->size(1);
  if (!optional(o[3], at::kFloat, T, k, w) || !optional(o[4], at::kBFloat16, T, y.cols, add)) Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_moe_combine)>(a.address(o[0]));
  void* stream = a.stream(o[5]);
  if (!a.ok || !here({y.t, slot, w.t, add.t})) Py_RETURN_NONE;
  const Fresh out(y.t, true, at::kBFloat16, {T, y.cols});
  return answer(entry(data<void>(y.t), type_of(f32), y.ld, y.rows, data<int32_t>(slot), data<float>(w.t), w.ld, T, k, y.cols,
                      data<void>(add.t), add.ld, out.data<void>(), y.cols, stream),
                out.t);
  END_HANDLE_TH_ERRORS
}

// moe_combine_bwd(entry, dout, slot, w, y, rows, codes, with_dy, out, stream)
// -> (q, s, dy, dw), a status, or None; rows None: as y has, or all
PyObject* moe_combine_bwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Matrix dout, w, y;
  bool f32 = false;
  const at::Tensor* slot;
  Numbers a;
  if (n != 10 || !matrix(o[1], at::kBFloat16, dout) || !slots(o[2], slot)) Py_RETURN_NONE;
  const int64_t T = dout.rows, k = slot->size(1), N = dout.cols;
  if (slot->size(0) != T || !matrix(o[3], at::kFloat, T, k, w)) Py_RETURN_NONE;
  if (o[4] != Py_None && (!values(o[4], y, f32) || y.cols != N)) Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_moe_combine_bwd)>(a.address(o[0]));
  const int64_t rows = o[5] != Py_None ? a.whole(o[5]) : y.t != nullptr ? y.rows : T * k;
  const bool with_q = a.flag(o[6]), with_dy = a.flag(o[7]), made = o[8] == Py_None;
  void* stream = a.stream(o[9]);
  if (!a.ok || rows < 0) Py_RETURN_NONE;
  Rows out(dout.t, made && with_q, made && with_dy, rows, N);
  if (!made && !out.take(o[8])) Py_RETURN_NONE;
  if (!here({dout.t, slot, w.t, y.t, out.mq.t, out.ms.t, out.my.t})) Py_RETURN_NONE;
  if (y.t != nullptr && y.rows != out.M) Py_RETURN_NONE;
  const Fresh dw(dout.t, y.t != nullptr, at::kFloat, {T, k});
  return answers(entry(data<void>(dout.t), dout.ld, data<void>(y.t), type_of(f32), y.ld, data<int32_t>(slot),
                       data<float>(w.t), w.ld, T, k, N, out.pq(), out.ldq(), out.ps(), out.lds(), out.py(), out.ldy(),
                       out.M, dw.data<float>(), k, stream),
                 {{out.given[0], out.q}, {out.given[1], out.s}, {out.given[2], out.y}, dw});
  END_HANDLE_TH_ERRORS
}

// swiglu_bwd_quant_1x128(entry, dh, g, u, codes, with_d, with_h, stream)
// -> (q, s, d, h), a status, or None
PyObject* swiglu_bwd_quant_1x128(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Matrix dh, g, u;
  Numbers a;
  if (n != 8 || !matrix(o[2], at::kBFloat16, g) || !matrix(o[1], at::kBFloat16, g.rows, g.cols, dh) ||
      !matrix(o[3], at::kBFloat16, g.rows, g.cols, u))
    Py_RETURN_NONE;
  const auto entry = reinterpret_cast<decltype(&fp8bs_swiglu_bwd_quant_1x128)>(a.address(o[0]));
  const bool with_q = a.flag(o[4]), with_d = a.flag(o[5]), with_h = a.flag(o[6]);
  void* stream = a.stream(o[7]);
  if (!a.ok || !here({dh.t, g.t, u.t})) Py_RETURN_NONE;
  const Rows out(g.t, with_q, with_d, g.rows, 2 * g.cols);
  const Fresh h(g.t, with_h, at::kBFloat16, {g.rows, g.cols});
  return answers(entry(data<void>(dh.t), dh.ld, data<void>(g.t), g.ld, data<void>(u.t), u.ld, g.rows, g.cols, out.pq(),
                       out.ldq(), out.ps(), out.lds(), out.py(), out.ldy(), h.data<void>(), g.cols, stream),
                 {out.q, out.s, out.y, h});
  END_HANDLE_TH_ERRORS
}

#define FP8BS_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP8BS_METHOD(rope), FP8BS_METHOD(kv_append), FP8BS_METHOD(attn_paged),
                         FP8BS_METHOD(rmsnorm_quant_1x128), FP8BS_METHOD(rmsnorm_bwd), FP8BS_METHOD(moe_dispatch),
                         FP8BS_METHOD(moe_combine), FP8BS_METHOD(moe_combine_bwd), FP8BS_METHOD(swiglu_bwd_quant_1x128),
                         {nullptr, nullptr, 0, nullptr}};
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
