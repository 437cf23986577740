// The Python binding's native half, for the operators between the GEMMs: a call's tensors (up to
// 18) are checked against the types, shapes, contiguity and device they must have and handed to the
// C entry point in one step. A forward norm's host time is 5.4 us, 3 of it the launch; with the same
// questions asked through the interpreter it was 17.
//
//   ptrs(spec, device, d0, d1, d2, *tensors) -> tuple of addresses, or the index of the first
//                                               tensor that is not as the specification says
//   bind(current stream, entry points' addresses)
//   ckpt_pack(x, q, s, pow2), ... -> the entry point's status, or None for arguments that are not
//                                    as they must be, which the binding then looks at one by one
//
// spec: four bytes per tensor: its type (b bf16, f fp32, q uint8), ! or ? (may be None, address 0),
// and the indices of its one or two sizes among d0, d1, d2 and the number 1 (3), - for none.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "puro.h"

namespace {

bool as_specified(const at::Tensor& t, const char* spec, int64_t device, const int64_t* dims) {
  const at::ScalarType type = spec[0] == 'b'   ? at::kBFloat16
                              : spec[0] == 'f' ? at::kFloat
                                               : at::kByte;
  const int64_t rank = spec[3] == '-' ? 1 : 2;
  if (t.scalar_type() != type || t.dim() != rank) return false;
  for (int64_t i = 0; i < rank; ++i)
    if (t.size(i) != dims[spec[2 + i] - '0']) return false;
  return t.is_contiguous() && t.is_cuda() && t.get_device() == device;
}

PyObject* ptrs(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t kFirst = 5;
  if (n < kFirst || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) != 4 * (n - kFirst)) {
    PyErr_SetString(PyExc_TypeError, "ptrs(spec, device, d0, d1, d2, *tensors)");
    return nullptr;
  }
  const char* spec = PyBytes_AS_STRING(args[0]);
  int64_t v[4];
  for (int i = 0; i < 4; ++i) v[i] = PyLong_AsLongLong(args[1 + i]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t dims[4] = {v[1], v[2], v[3], 1};
  PyObject* out = PyTuple_New(n - kFirst);
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 0; i < n - kFirst; ++i, spec += 4) {
    PyObject* o = args[kFirst + i];
    uint64_t address = 0;
    bool ok = o == Py_None ? spec[1] == '?' : false;
    if (!ok && THPVariable_Check(o)) {
      try {
        const at::Tensor& t = THPVariable_Unpack(o);
        ok = as_specified(t, spec, v[0], dims);
        if (ok) address = reinterpret_cast<uint64_t>(t.const_data_ptr());
      } catch (const std::exception&) {  // a layout without strides or storage (sparse, nested)
        ok = false;
      }
    }
    PyObject* item = ok ? PyLong_FromUnsignedLongLong(address) : nullptr;
    if (item == nullptr) {
      Py_DECREF(out);
      return PyErr_Occurred() ? nullptr : PyLong_FromSsize_t(i);
    }
    PyTuple_SET_ITEM(out, i, item);
  }
  return out;
}

// ---------------------------------------------------------------- whole calls
struct Entries {
  PyObject* stream;   // device index -> raw handle of torch's current stream
  decltype(&puro_ckpt_pack) pack;
  decltype(&puro_ckpt_unpack) unpack;
  decltype(&puro_ckpt_transpose) transpose;
  decltype(&puro_block_norm_fwd) norm_fwd;
  decltype(&puro_block_norm_workspace) norm_workspace;
  decltype(&puro_block_norm_bwd) norm_bwd;
  decltype(&puro_swiglu_fwd) swiglu_fwd;
  decltype(&puro_swiglu_bwd) swiglu_bwd;
  decltype(&puro_swiglu_bwd_fp8) swiglu_bwd_fp8;
  decltype(&puro_linear_xent_fwd_workspace) xent_fwd_workspace;
  decltype(&puro_linear_xent_fwd) xent_fwd;
  decltype(&puro_linear_xent_bwd_workspace) xent_bwd_workspace;
  decltype(&puro_linear_xent_bwd) xent_bwd;
  decltype(&puro_newton_schulz_workspace) ns_workspace;
  decltype(&puro_newton_schulz) ns;
} entry = {};

template <typename F>
bool take_address(PyObject* o, F* f) {
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  *f = reinterpret_cast<F>(static_cast<uintptr_t>(v));
  return v != 0 && !PyErr_Occurred();
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Entries e = {};
  if (n != 16 || !take_address(a[1], &e.pack) || !take_address(a[2], &e.unpack) ||
      !take_address(a[3], &e.transpose) || !take_address(a[4], &e.norm_fwd) ||
      !take_address(a[5], &e.norm_workspace) || !take_address(a[6], &e.norm_bwd) ||
      !take_address(a[7], &e.swiglu_fwd) || !take_address(a[8], &e.swiglu_bwd) ||
      !take_address(a[9], &e.swiglu_bwd_fp8) || !take_address(a[10], &e.xent_fwd_workspace) ||
      !take_address(a[11], &e.xent_fwd) || !take_address(a[12], &e.xent_bwd_workspace) ||
      !take_address(a[13], &e.xent_bwd) || !take_address(a[14], &e.ns_workspace) ||
      !take_address(a[15], &e.ns)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "bind(stream, fifteen addresses)");
    return nullptr;
  }
  e.stream = Py_NewRef(a[0]);
  Py_XSETREF(entry.stream, e.stream);
  entry = e;
  Py_RETURN_NONE;
}

const at::Tensor* as_tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// The tensors of one call: all on the device of the first, `ok` until one is not as it must be.
struct Call {
  const at::Tensor* lead;
  int64_t rows = 0, cols = 0, device = -1;
  bool ok;
  // A matrix that gives the call its sizes and device.
  explicit Call(PyObject* o) : lead(as_tensor(o)) {
    ok = lead != nullptr && lead->dim() == 2 && lead->is_cuda();
    if (!ok) return;
    rows = lead->size(0), cols = lead->size(1), device = lead->get_device();
  }
  // Address of a contiguous tensor [d0][d1] (d1 < 0: [d0]).
  template <typename T = void>
  T* get(PyObject* o, at::ScalarType type, int64_t d0, int64_t d1) {
    const at::Tensor* t = ok ? as_tensor(o) : nullptr;
    ok = t != nullptr && t->scalar_type() == type && t->dim() == (d1 < 0 ? 1 : 2) &&
         t->size(0) == d0 && (d1 < 0 || t->size(1) == d1) && t->is_contiguous() && t->is_cuda() &&
         t->get_device() == device;
    return ok ? static_cast<T*>(const_cast<void*>(t->const_data_ptr())) : nullptr;
  }
  template <typename T = void>
  T* may(PyObject* o, at::ScalarType type, int64_t d0, int64_t d1) {
    return o == Py_None ? nullptr : get<T>(o, type, d0, d1);
  }
  // The 16- or 32-bit side of a checkpoint: adjacent columns, any row stride from cols up.
  void* wide(const at::Tensor* t, int* type, int64_t* ld) {
    ok = ok && t != nullptr && t->layout() == at::kStrided && t->dim() == 2 &&
         t->size(0) == rows && t->size(1) == cols && t->is_cuda() && t->get_device() == device &&
         (t->scalar_type() == at::kBFloat16 || t->scalar_type() == at::kFloat);
    if (!ok) return nullptr;
    *type = t->scalar_type() == at::kFloat ? PURO_TYPE_FP32 : PURO_TYPE_BF16;
    *ld = rows <= 1 ? cols : t->stride(0);
    ok = (cols <= 1 || t->stride(1) == 1) && *ld >= cols;
    return ok ? const_cast<void*>(t->const_data_ptr()) : nullptr;
  }
  // A saved activation as it was or as a (codes, scales) pair: `s0` groups of columns.
  void saved(PyObject* o, at::ScalarType type, int64_t d1, int64_t s0, const void** x,
             const void** q, const float** s) {
    if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2) {
      *q = get(PyTuple_GET_ITEM(o, 0), at::kByte, rows, d1);
      *s = get<float>(PyTuple_GET_ITEM(o, 1), at::kFloat, s0, rows);
    } else {
      *x = get(o, type, rows, d1);
    }
  }
  double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int flag(PyObject* o) {
    ok = ok && PyBool_Check(o);
    return o == Py_True;
  }
  void* stream() {
    PyObject* d = PyLong_FromLongLong(device);
    PyObject* h = d != nullptr ? PyObject_CallOneArg(entry.stream, d) : nullptr;
    void* p = h != nullptr ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(d);
    Py_XDECREF(h);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return p;
  }
};

// Calls f(stream) without the interpreter's lock; None if the arguments were not in order.
template <typename F>
PyObject* finish(Call& c, F&& f) {
  if (!c.ok) Py_RETURN_NONE;
  // the tensors' device may not be the current one, which launches (and the default stream) go by
  const c10::DeviceGuard guard(c.lead->device());
  void* stream = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  puro_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f(stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

int64_t groups(int64_t n) { return (n + 127) / 128; }
bool outputs(PyObject* o, Py_ssize_t n) { return PyTuple_Check(o) && PyTuple_GET_SIZE(o) == n; }

PyObject* ckpt_pack(PyObject* const* a) {   // x, q, s, pow2
  Call c(a[0]);
  int type = 0;
  int64_t ld = 0;
  const void* x = c.wide(c.lead, &type, &ld);
  void* q = c.get(a[1], at::kByte, c.rows, c.cols);
  float* s = c.get<float>(a[2], at::kFloat, groups(c.cols), c.rows);
  const int pow2 = c.flag(a[3]);
  return finish(c, [&](void* st) {
    return entry.pack(x, type, c.rows, c.cols, ld, pow2, q, s, st);
  });
}

PyObject* ckpt_unpack(PyObject* const* a) {   // q, s, x
  Call c(a[0]);
  const void* q = c.get(a[0], at::kByte, c.rows, c.cols);
  const float* s = c.get<float>(a[1], at::kFloat, groups(c.cols), c.rows);
  int type = 0;
  int64_t ld = 0;
  void* x = c.wide(as_tensor(a[2]), &type, &ld);
  return finish(c, [&](void* st) { return entry.unpack(q, s, c.rows, c.cols, x, type, ld, st); });
}

PyObject* ckpt_transpose(PyObject* const* a) {   // q, s, qt, st, pow2
  Call c(a[0]);
  const void* q = c.get(a[0], at::kByte, c.rows, c.cols);
  const float* s = c.get<float>(a[1], at::kFloat, groups(c.cols), c.rows);
  void* qt = c.get(a[2], at::kByte, c.cols, c.rows);
  float* ts = c.get<float>(a[3], at::kFloat, groups(c.rows), c.cols);
  const int pow2 = c.flag(a[4]);
  return finish(c, [&](void* st) {
    return entry.transpose(q, s, c.rows, c.cols, pow2, qt, ts, st);
  });
}

// A gate's kind, and its address (of a gradient: the same form).
int gate_kind(PyObject* o) {
  const at::Tensor* t = as_tensor(o);
  if (t == nullptr) return PURO_GATE_NONE;
  if (t->dim() == 1) return PURO_GATE_CHANNEL;
  return t->scalar_type() == at::kFloat ? PURO_GATE_TOKEN : PURO_GATE_FULL;
}
void* gate(Call& c, PyObject* o, int kind) {
  switch (kind) {
    case PURO_GATE_CHANNEL: return c.get(o, at::kFloat, c.cols, -1);
    case PURO_GATE_TOKEN: return c.get(o, at::kFloat, c.rows, 1);
    case PURO_GATE_FULL: return c.get(o, at::kBFloat16, c.rows, c.cols);
    default: c.ok = c.ok && o == Py_None; return nullptr;
  }
}
bool residual(Call& c, at::ScalarType type) {
  c.ok = c.ok && (type == at::kBFloat16 || type == at::kFloat);
  return type == at::kFloat;
}

PyObject* norm_fwd(PyObject* const* a) {
  // y, r, w_post, w_pre, gate, alpha, beta, eps, pow2, (r_out, n, nq, ns, rstd_y, rstd_r, yq, ys,
  // rq, rs)
  Call c(a[1]);
  if (!c.ok || !outputs(a[9], 10)) Py_RETURN_NONE;
  const at::ScalarType res = c.lead->scalar_type();
  puro_block_norm d = {};
  d.residual_type = residual(c, res) ? PURO_TYPE_FP32 : PURO_TYPE_BF16;
  const int64_t rows = d.rows = c.rows, cols = d.cols = c.cols, k = groups(cols);
  d.gate_kind = gate_kind(a[4]);
  d.alpha = static_cast<float>(c.number(a[5]));
  d.beta = static_cast<float>(c.number(a[6]));
  d.eps = static_cast<float>(c.number(a[7]));
  d.pow2 = c.flag(a[8]);
  d.y = c.may(a[0], at::kBFloat16, rows, cols);
  d.r = c.get(a[1], res, rows, cols);
  d.w_post = a[0] == Py_None ? nullptr : c.may<float>(a[2], at::kFloat, cols, -1);
  d.w_pre = c.may<float>(a[3], at::kFloat, cols, -1);
  d.gate = gate(c, a[4], d.gate_kind);
  PyObject* const* o = &PyTuple_GET_ITEM(a[9], 0);
  d.r_out = c.may(o[0], res, rows, cols);
  d.n = c.may(o[1], at::kBFloat16, rows, cols);
  d.nq = c.may(o[2], at::kByte, rows, cols);
  d.ns = c.may<float>(o[3], at::kFloat, k, rows);
  d.rstd_y = c.may<float>(o[4], at::kFloat, rows, -1);
  d.rstd_r = c.may<float>(o[5], at::kFloat, rows, -1);
  d.yq = c.may(o[6], at::kByte, rows, cols);
  d.ys = c.may<float>(o[7], at::kFloat, k, rows);
  d.rq = c.may(o[8], at::kByte, rows, cols);
  d.rs = c.may<float>(o[9], at::kFloat, k, rows);
  return finish(c, [&](void* st) { return entry.norm_fwd(&d, st); });
}

PyObject* norm_bwd(PyObject* const* a) {
  // dr_out, dn, y, r_out, rstd_y, rstd_r, w_post, w_pre, gate, alpha, beta, accumulate, workspace,
  // (dr, dy, dw_post, dw_pre, dgate)
  Call c(a[0] != Py_None ? a[0] : a[1]);
  if (!c.ok || !outputs(a[13], 5)) Py_RETURN_NONE;
  PyObject* const* o = &PyTuple_GET_ITEM(a[13], 0);
  const bool post = a[4] != Py_None, pre = a[1] != Py_None;
  // the residual type: that of dr_out, else of r_out, else of dr; without any of them nothing of
  // that type is read or written
  const at::Tensor* typed = a[0] != Py_None ? c.lead : as_tensor(a[3]);
  if (typed == nullptr) typed = as_tensor(o[0]);
  const at::ScalarType res = typed != nullptr ? typed->scalar_type() : at::kBFloat16;
  puro_block_norm_grad d = {};
  d.residual_type = residual(c, res) ? PURO_TYPE_FP32 : PURO_TYPE_BF16;
  const int64_t rows = d.rows = c.rows, cols = d.cols = c.cols, k = groups(cols);
  d.gate_kind = gate_kind(a[8]);
  d.alpha = static_cast<float>(c.number(a[9]));
  d.beta = static_cast<float>(c.number(a[10]));
  d.accumulate = c.flag(a[11]);
  d.dr_out = c.may(a[0], res, rows, cols);
  d.dn = c.may(a[1], at::kBFloat16, rows, cols);
  if (post) {
    c.saved(a[2], at::kBFloat16, cols, k, &d.y, &d.yq, &d.ys);
    d.rstd_y = c.get<float>(a[4], at::kFloat, rows, -1);
    d.w_post = c.may<float>(a[6], at::kFloat, cols, -1);
  }
  if (pre) {
    c.saved(a[3], res, cols, k, &d.r, &d.rq, &d.rs);
    d.rstd_r = c.may<float>(a[5], at::kFloat, rows, -1);
    d.w_pre = c.may<float>(a[7], at::kFloat, cols, -1);
  }
  d.gate = gate(c, a[8], d.gate_kind);
  d.dr = c.may(o[0], res, rows, cols);
  d.dy = c.may(o[1], at::kBFloat16, rows, cols);
  d.dw_post = c.may<float>(o[2], at::kFloat, cols, -1);
  d.dw_pre = c.may<float>(o[3], at::kFloat, cols, -1);
  d.dgate = gate(c, o[4], d.gate_kind);
  if (!c.ok) Py_RETURN_NONE;
  const int64_t need = entry.norm_workspace(rows, cols);
  at::Tensor own;
  const at::Tensor* w = as_tensor(a[12]);
  if (a[12] == Py_None) {   // from torch's allocator, in the order of the current stream
    own = at::empty({need > 16 ? need : 16}, c.lead->options().dtype(at::kByte));
    w = &own;
  }
  // contiguous: a view's elements may share their bytes, or lie apart
  c.ok = w != nullptr && w->is_cuda() && w->get_device() == c.device && w->is_contiguous() &&
         static_cast<int64_t>(w->numel() * w->element_size()) >= need;
  void* ws = c.ok ? const_cast<void*>(w->const_data_ptr()) : nullptr;
  return finish(c, [&](void* st) { return entry.norm_bwd(&d, ws, st); });
}

PyObject* swiglu_fwd(PyObject* const* a) {   // gu, pow2, (h, hq, hs, guq, gus)
  Call c(a[0]);
  if (!c.ok || c.cols % 2 != 0 || !outputs(a[2], 5)) Py_RETURN_NONE;
  const int64_t rows = c.rows, f = c.cols / 2, k = groups(f);
  PyObject* const* o = &PyTuple_GET_ITEM(a[2], 0);
  const void* gu = c.get(a[0], at::kBFloat16, rows, 2 * f);
  void* h = c.may(o[0], at::kBFloat16, rows, f);
  void* hq = c.may(o[1], at::kByte, rows, f);
  float* hs = c.may<float>(o[2], at::kFloat, k, rows);
  void* guq = c.may(o[3], at::kByte, rows, 2 * f);
  float* gus = c.may<float>(o[4], at::kFloat, 2 * k, rows);
  const int pow2 = c.flag(a[1]);
  return finish(c, [&](void* st) {
    return entry.swiglu_fwd(gu, rows, f, h, hq, hs, guq, gus, pow2, st);
  });
}

PyObject* swiglu_bwd(PyObject* const* a) {   // dh, gu, dgu
  Call c(a[0]);
  const int64_t rows = c.rows, f = c.cols;
  const void *gu = nullptr, *guq = nullptr;
  const float* gus = nullptr;
  const void* dh = c.get(a[0], at::kBFloat16, rows, f);
  c.saved(a[1], at::kBFloat16, 2 * f, 2 * groups(f), &gu, &guq, &gus);
  void* dgu = c.get(a[2], at::kBFloat16, rows, 2 * f);
  return finish(c, [&](void* st) {
    return entry.swiglu_bwd(dh, gu, guq, gus, rows, f, dgu, st);
  });
}

PyObject* swiglu_bwd_fp8(PyObject* const* a) {
  // dh, gu, pow2, (dguq, dgus, dgutq, dguts, htq, hts)
  Call c(a[0]);
  if (!c.ok || c.rows % 128 != 0 || c.cols % 128 != 0 || !outputs(a[3], 6)) Py_RETURN_NONE;
  const int64_t rows = c.rows, f = c.cols;
  PyObject* const* o = &PyTuple_GET_ITEM(a[3], 0);
  const void *gu = nullptr, *guq = nullptr;
  const float* gus = nullptr;
  const void* dh = c.get(a[0], at::kBFloat16, rows, f);
  c.saved(a[1], at::kBFloat16, 2 * f, f / 64, &gu, &guq, &gus);
  const int pow2 = c.flag(a[2]);
  void* dguq = c.get(o[0], at::kByte, rows, 2 * f);
  float* dgus = c.get<float>(o[1], at::kFloat, f / 64, rows);
  void* dgutq = c.get(o[2], at::kByte, 2 * f, rows);
  float* dguts = c.get<float>(o[3], at::kFloat, rows / 128, 2 * f);
  void* htq = c.get(o[4], at::kByte, f, rows);
  float* hts = c.get<float>(o[5], at::kFloat, rows / 128, f);
  return finish(c, [&](void* st) {
    return entry.swiglu_bwd_fp8(dh, gu, guq, gus, rows, f, pow2, dguq, dgus, dgutq, dguts, htq, hts,
                                st);
  });
}

// The caller's scratch memory of at least `need` bytes, or (None) some of torch's, in the order of the
// current stream.
void* scratch(Call& c, PyObject* o, int64_t need, at::Tensor* own) {
  if (!c.ok) return nullptr;
  const at::Tensor* w = as_tensor(o);
  if (o == Py_None) {
    *own = at::empty({need}, c.lead->options().dtype(at::kByte));
    w = own;
  }
  c.ok = w != nullptr && w->layout() == at::kStrided && w->is_contiguous() && w->is_cuda() &&
         w->get_device() == c.device && w->numel() * static_cast<int64_t>(w->element_size()) >= need;
  return c.ok ? const_cast<void*>(w->const_data_ptr()) : nullptr;
}

// A bf16 matrix of `cols` adjacent columns and any row stride from cols up.
const void* bf16_rows(Call& c, const at::Tensor* t, int64_t cols, int64_t* rows, int64_t* ld) {
  c.ok = c.ok && t != nullptr && t->layout() == at::kStrided && t->dim() == 2 &&
         t->scalar_type() == at::kBFloat16 && t->size(1) == cols && t->is_cuda() &&
         t->get_device() == c.device;
  if (!c.ok) return nullptr;
  *rows = t->size(0);
  *ld = *rows <= 1 ? cols : t->stride(0);
  c.ok = (cols <= 1 || t->stride(1) == 1) && *ld >= cols;
  return c.ok ? t->const_data_ptr() : nullptr;
}

PyObject* xent_fwd(PyObject* const* a) {   // h, w, targets, loss, lse, workspace
  Call c(a[0]);
  puro_linear_xent d = {};
  d.d = c.cols;
  d.h = bf16_rows(c, c.lead, d.d, &d.tokens, &d.ldh);
  d.w = c.ok ? bf16_rows(c, as_tensor(a[1]), d.d, &d.vocab, &d.ldw) : nullptr;
  d.targets = c.get<int64_t>(a[2], at::kLong, d.tokens, -1);
  d.loss = c.get<float>(a[3], at::kFloat, d.tokens, -1);
  d.lse = c.get<float>(a[4], at::kFloat, d.tokens, -1);
  at::Tensor own;
  void* ws = c.ok ? scratch(c, a[5], entry.xent_fwd_workspace(&d), &own) : nullptr;
  return finish(c, [&](void* st) { return entry.xent_fwd(&d, ws, st); });
}

PyObject* xent_bwd(PyObject* const* a) {
  // h, w, targets, lse, dloss, dlse, dh, dw, accumulate, workspace
  Call c(a[0]);
  puro_linear_xent_grad d = {};
  d.d = c.cols;
  d.h = bf16_rows(c, c.lead, d.d, &d.tokens, &d.ldh);
  d.w = c.ok ? bf16_rows(c, as_tensor(a[1]), d.d, &d.vocab, &d.ldw) : nullptr;
  d.targets = c.get<int64_t>(a[2], at::kLong, d.tokens, -1);
  d.lse = c.get<float>(a[3], at::kFloat, d.tokens, -1);
  d.dloss = c.get<float>(a[4], at::kFloat, d.tokens, -1);
  d.dlse = c.may<float>(a[5], at::kFloat, d.tokens, -1);
  d.dh = c.may(a[6], at::kBFloat16, d.tokens, d.d);
  const at::Tensor* dw = c.ok && a[7] != Py_None ? as_tensor(a[7]) : nullptr;
  const bool f32 = dw != nullptr && dw->scalar_type() == at::kFloat;
  d.dw_type = f32 ? PURO_TYPE_FP32 : PURO_TYPE_BF16;
  d.dw = c.may(a[7], f32 ? at::kFloat : at::kBFloat16, d.vocab, d.d);
  d.accumulate = c.flag(a[8]);
  at::Tensor own;
  void* ws = c.ok ? scratch(c, a[9], entry.xent_bwd_workspace(&d), &own) : nullptr;
  return finish(c, [&](void* st) { return entry.xent_bwd(&d, ws, st); });
}

PyObject* newton_schulz(PyObject* const* a) {
  // [g], [m] or None, [m_out] (None with m), [u], beta, nesterov, scale, steps, (coefficients),
  // workspace
  const bool momentum = a[1] != Py_None;
  if (!PyList_Check(a[0]) || !PyList_Check(a[3]) || (momentum && !PyList_Check(a[1])) ||
      (momentum && !PyList_Check(a[2])) || !PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 3 ||
      !PyLong_Check(a[7]))
    Py_RETURN_NONE;
  const Py_ssize_t n = PyList_GET_SIZE(a[0]);
  if (n < 1 || n > PURO_NS_GROUP_MAX || PyList_GET_SIZE(a[3]) != n ||
      (momentum && (PyList_GET_SIZE(a[1]) != n || PyList_GET_SIZE(a[2]) != n)))
    Py_RETURN_NONE;
  Call c(PyList_GET_ITEM(a[0], 0));
  puro_ns_item items[PURO_NS_GROUP_MAX] = {};
  for (Py_ssize_t i = 0; i < n && c.ok; ++i) {
    items[i].g = c.get<float>(PyList_GET_ITEM(a[0], i), at::kFloat, c.rows, c.cols);
    if (momentum) {
      items[i].m = c.get<float>(PyList_GET_ITEM(a[1], i), at::kFloat, c.rows, c.cols);
      items[i].m_out = c.get<float>(PyList_GET_ITEM(a[2], i), at::kFloat, c.rows, c.cols);
    }
    items[i].u = c.get(PyList_GET_ITEM(a[3], i), at::kBFloat16, c.rows, c.cols);
  }
  puro_newton_schulz_params h = {};
  h.beta = static_cast<float>(c.number(a[4]));
  h.nesterov = c.flag(a[5]);
  h.scale = static_cast<float>(c.number(a[6]));
  const long steps = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) PyErr_Clear();
  c.ok = c.ok && steps >= 1 && steps <= PURO_NS_MAX_STEPS;
  h.steps = static_cast<int>(steps);
  for (int i = 0; i < 3; ++i)
    h.coefficients[i] = static_cast<float>(c.number(PyTuple_GET_ITEM(a[8], i)));
  at::Tensor own;
  void* ws = c.ok ? scratch(c, a[9], entry.ns_workspace(n, c.rows, c.cols), &own) : nullptr;
  return finish(c, [&](void* st) {
    return entry.ns(items, static_cast<int>(n), c.rows, c.cols, &h, ws, st);
  });
}

// As a method of kN arguments; torch's exceptions (a layout without strides or storage) and a
// wrong number of arguments leave the question to the binding.
template <PyObject* (*kCall)(PyObject* const*), Py_ssize_t kN>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kN || entry.stream == nullptr) Py_RETURN_NONE;
  try {
    return kCall(a);
  } catch (const std::exception&) {
    Py_RETURN_NONE;
  }
}
template <typename F>
PyCFunction as_method(F* f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef kMethods[] = {
    {"ptrs", as_method(ptrs), METH_FASTCALL, "Checked addresses of an operator's tensors."},
    {"bind", as_method(bind), METH_FASTCALL, "Sets the C entry points."},
    {"ckpt_pack", as_method(method<ckpt_pack, 4>), METH_FASTCALL, nullptr},
    {"ckpt_unpack", as_method(method<ckpt_unpack, 3>), METH_FASTCALL, nullptr},
    {"ckpt_transpose", as_method(method<ckpt_transpose, 5>), METH_FASTCALL, nullptr},
    {"norm_fwd", as_method(method<norm_fwd, 10>), METH_FASTCALL, nullptr},
    {"norm_bwd", as_method(method<norm_bwd, 14>), METH_FASTCALL, nullptr},
    {"swiglu_fwd", as_method(method<swiglu_fwd, 3>), METH_FASTCALL, nullptr},
    {"swiglu_bwd", as_method(method<swiglu_bwd, 3>), METH_FASTCALL, nullptr},
    {"swiglu_bwd_fp8", as_method(method<swiglu_bwd_fp8, 4>), METH_FASTCALL, nullptr},
    {"xent_fwd", as_method(method<xent_fwd, 6>), METH_FASTCALL, nullptr},
    {"xent_bwd", as_method(method<xent_bwd, 10>), METH_FASTCALL, nullptr},
    {"newton_schulz", as_method(method<newton_schulz, 10>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_args", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args(void) { return PyModule_Create(&kModule); }
