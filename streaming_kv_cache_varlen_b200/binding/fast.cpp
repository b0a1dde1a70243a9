// The usual calls of the paged cache operators without the interpreter: arguments
// checked, outputs allocated and the C entry point called in one step (1 to 2 us
// beside the launches, where the Python path takes 8 to 15 us; a decode step's append
// runs 5 us on the device).
//
// A function here takes exactly the calls that the Python functions of the package
// would pass on: tensors of the right types and shapes on the current device, on its
// current stream. For anything else it does nothing and returns -1, and the Python
// path then says what is wrong (or handles it: another device or stream). Other
// integers are statuses of the C call.
#include <Python.h>

#include <cmath>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "cmp.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* status(long s) { return PyLong_FromLong(s); }

// A tensor argument, or null.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Call {
  int dev;
  ScalarType dtype;
  int32_t dt;

  // q or k: fixes the device and the element type of the call
  bool begin(const Tensor* t) {
    if (!t || !t->is_cuda() || t->dim() != 3) return false;
    dev = t->device().index();
    dtype = t->scalar_type();
    if (dtype == ScalarType::Half) dt = CMP_NSA_FP16;
    else if (dtype == ScalarType::BFloat16) dt = CMP_NSA_BF16;
    else return false;
    return c10::cuda::current_device() == dev;
  }
  bool here(const Tensor* t, ScalarType s, int64_t dim) const {
    return t && t->is_cuda() && t->scalar_type() == s && t->device().index() == dev && t->dim() == dim;
  }
  bool dense(const Tensor* t, ScalarType s, int64_t dim) const { return here(t, s, dim) && t->is_contiguous(); }
  // [T, H, D] with the last two dimensions dense: its token stride
  bool tokens(const Tensor* t, int64_t T, int64_t H, int64_t D, int64_t* stride) const {
    if (!here(t, dtype, 3) || t->size(0) != T || t->size(1) != H || t->size(2) != D) return false;
    if ((D > 1 && t->stride(2) != 1) || (H > 1 && t->stride(1) != D)) return false;
    *stride = T <= 1 ? H * D : t->stride(0);
    return *stride >= H * D && *stride % 8 == 0 && reinterpret_cast<uintptr_t>(t->data_ptr()) % 16 == 0;
  }
  bool weight(const Tensor* t, int64_t D) const { return dense(t, dtype, 1) && t->size(0) == D; }
  // 0: no rotation, 1: in r, -1: not a call for here
  int rope(PyObject* sin, PyObject* cos, PyObject* pairs, int64_t T, int64_t D, cmp_rope* r) const {
    if (!PyUnicode_Check(pairs)) return -1;
    if (PyUnicode_CompareWithASCIIString(pairs, "interleaved") == 0) r->pairs = CMP_ROPE_INTERLEAVED;
    else if (PyUnicode_CompareWithASCIIString(pairs, "halves") == 0) r->pairs = CMP_ROPE_HALVES;
    else return -1;
    if (sin == Py_None && cos == Py_None) return 0;
    const Tensor *s = tensor(sin), *c = tensor(cos);
    if (!s || !c) return -1;
    const ScalarType t = s->scalar_type();
    if (t != ScalarType::Float && t != ScalarType::BFloat16) return -1;
    if (!dense(s, t, 2) || !dense(c, t, 2)) return -1;
    const int64_t R = s->size(1);
    if (s->size(0) != T || c->size(0) != T || c->size(1) != R || R < 16 || R % 16 || R > D) return -1;
    r->sin = s->data_ptr();
    r->cos = c->data_ptr();
    r->dim = (int32_t)R;
    r->dtype = t == ScalarType::Float ? CMP_ROPE_F32 : CMP_ROPE_BF16;
    return 1;
  }
  bool caches(const Tensor* k, const Tensor* v, int64_t Hk, int64_t D) const {
    return dense(k, dtype, 4) && dense(v, dtype, 4) && k->sizes() == v->sizes() && k->size(2) == Hk && k->size(3) == D;
  }
  // B, or -1
  int64_t sequences(const Tensor* table, const Tensor* cu, PyObject* start, const int32_t** start_ptr) const {
    if (!dense(table, ScalarType::Int, 2) || !dense(cu, ScalarType::Int, 1)) return -1;
    const int64_t B = cu->size(0) - 1;
    if (B < 0 || table->size(0) != B) return -1;
    *start_ptr = nullptr;
    if (start != Py_None) {
      const Tensor* s = tensor(start);
      if (!dense(s, ScalarType::Int, 1) || s->size(0) != B) return -1;
      *start_ptr = static_cast<const int32_t*>(s->data_ptr());
    }
    return B;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

const int32_t* ints(const Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); }

// A float argument (a Python float or int).
bool number(PyObject* o, float* f) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  const double d = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *f = (float)d;
  return true;
}

// An int argument of at least lo; None: 0.
bool integer(PyObject* o, int64_t lo, int64_t* v) {
  *v = 0;
  if (o == Py_None) return true;
  if (!PyLong_Check(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return *v >= lo;
}

// q, k, q_weight, k_weight, sin, cos, rope_pairs, eps, q_out, k_out -> (q_out, k_out) or a status
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) return status(-1);
  Call c;
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *qw = tensor(a[2]), *kw = tensor(a[3]);
  if (!c.begin(q)) return status(-1);
  cmp_qk_dims d{};
  d.T = q->size(0);
  d.Hq = q->size(1);
  d.D = q->size(2);
  float eps;
  if (!c.tokens(q, d.T, d.Hq, d.D, &d.q_stride) || !c.weight(qw, d.D) || !number(a[7], &eps)) return status(-1);
  if (a[1] != Py_None) {
    if (!k || k->dim() != 3) return status(-1);
    d.Hk = k->size(1);
    if (!c.tokens(k, d.T, d.Hk, d.D, &d.k_stride) || !c.weight(kw, d.D)) return status(-1);
  }
  cmp_rope rope{};
  const int rot = c.rope(a[4], a[5], a[6], d.T, d.D, &rope);
  if (rot < 0) return status(-1);
  const Tensor *qo = tensor(a[8]), *ko = tensor(a[9]);
  Tensor q_new, k_new;
  if (a[8] == Py_None) {
    q_new = at::empty({d.T, d.Hq, d.D}, q->options());
    qo = &q_new;
  }
  if (!c.tokens(qo, d.T, d.Hq, d.D, &d.q_out_stride)) return status(-1);
  if (k) {
    if (a[9] == Py_None) {
      k_new = at::empty({d.T, d.Hk, d.D}, q->options());
      ko = &k_new;
    }
    if (!c.tokens(ko, d.T, d.Hk, d.D, &d.k_out_stride)) return status(-1);
  }
  const int st = cmp_qk_norm_rope(q->data_ptr(), k ? k->data_ptr() : nullptr, qw->data_ptr(),
                                  k ? kw->data_ptr() : nullptr, rot ? &rope : nullptr, eps, c.dt, qo->data_ptr(),
                                  k ? ko->data_ptr() : nullptr, c.stream(), &d);
  if (st != CMP_OK) return status(st);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyObject* x = THPVariable_Wrap(*qo);
  PyObject* y = k ? THPVariable_Wrap(*ko) : Py_NewRef(Py_None);
  PyTuple_SET_ITEM(r, 0, x);
  PyTuple_SET_ITEM(r, 1, y);
  return r;
}

// k, v, k_cache, v_cache, block_table, cu_seqlens, start_pos, norm_weight, sin, cos, rope_pairs, eps -> status
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return status(-1);
  Call c;
  const Tensor *k = tensor(a[0]), *v = tensor(a[1]), *kc = tensor(a[2]), *vc = tensor(a[3]), *table = tensor(a[4]),
               *cu = tensor(a[5]), *w = tensor(a[7]);
  if (!c.begin(k)) return status(-1);
  cmp_kv_dims d{};
  d.T = k->size(0);
  d.Hk = k->size(1);
  d.D = k->size(2);
  float eps;
  const int32_t* start;
  if (!c.tokens(k, d.T, d.Hk, d.D, &d.k_stride) || !c.tokens(v, d.T, d.Hk, d.D, &d.v_stride) ||
      !c.caches(kc, vc, d.Hk, d.D) || (d.B = c.sequences(table, cu, a[6], &start)) < 0 ||
      (a[7] != Py_None && !c.weight(w, d.D)) || !number(a[11], &eps))
    return status(-1);
  cmp_rope rope{};
  const int rot = c.rope(a[8], a[9], a[10], d.T, d.D, &rope);
  if (rot < 0) return status(-1);
  d.block_num = kc->size(0);
  d.page_size = kc->size(1);
  d.table_stride = table->size(1);
  return status(cmp_kv_append(k->data_ptr(), v->data_ptr(), a[7] == Py_None ? nullptr : w->data_ptr(),
                              rot ? &rope : nullptr, eps, ints(table), ints(cu), start, c.dt, kc->data_ptr(),
                              vc->data_ptr(), c.stream(), &d));
}

// q, k_cache, v_cache, block_table, cu_seqlens, start_pos, scale, max_len, window, key_block, key_stride, out, lse,
// return_lse, workspace -> out, (out, lse) or a status
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15) return status(-1);
  Call c;
  const Tensor *q = tensor(a[0]), *kc = tensor(a[1]), *vc = tensor(a[2]), *table = tensor(a[3]), *cu = tensor(a[4]),
               *out = tensor(a[11]), *lse = tensor(a[12]), *ws = tensor(a[14]);
  if (!c.begin(q) || !kc || kc->dim() != 4) return status(-1);
  cmp_attn_dims d{};
  d.T = q->size(0);
  d.Hq = q->size(1);
  d.D = q->size(2);
  d.Hk = kc->size(2);
  const int32_t* start;
  int64_t window, key_block, key_stride;
  float scale = (float)std::pow((double)d.D, -0.5);
  if (!c.tokens(q, d.T, d.Hq, d.D, &d.q_stride) || !c.caches(kc, vc, d.Hk, d.D) ||
      (d.B = c.sequences(table, cu, a[5], &start)) < 0 || (a[6] != Py_None && !number(a[6], &scale)) ||
      !integer(a[7], 1, &d.max_len) || !integer(a[8], 1, &window) || a[9] == Py_None || a[10] == Py_None ||
      !integer(a[9], 1, &key_block) || !integer(a[10], 1, &key_stride))
    return status(-1);
  d.block_num = kc->size(0);
  d.page_size = kc->size(1);
  d.table_stride = table->size(1);
  const int asked = PyObject_IsTrue(a[13]);  // any truth value, as in the Python path
  if (asked < 0) {
    PyErr_Clear();
    return status(-1);
  }
  const bool want_lse = a[12] != Py_None || asked;
  Tensor out_new, lse_new, ws_new;
  if (a[11] != Py_None &&
      (!c.dense(out, c.dtype, 3) || out->size(0) != d.T || out->size(1) != d.Hq || out->size(2) != d.D))
    return status(-1);
  if (a[12] != Py_None && (!c.dense(lse, ScalarType::Float, 2) || lse->size(0) != d.T || lse->size(1) != d.Hq))
    return status(-1);
  size_t have;
  if (a[14] == Py_None) {
    have = cmp_paged_attention_workspace(&d);
    if (have == 0) return status(CMP_ERR_INVALID);
    ws_new = at::empty({(int64_t)have}, q->options().dtype(ScalarType::Byte));
    ws = &ws_new;
  } else {
    if (!ws || !ws->is_cuda() || ws->device().index() != c.dev || !ws->is_contiguous()) return status(-1);
    have = ws->nbytes();
  }
  if (a[11] == Py_None) {
    out_new = at::empty({d.T, d.Hq, d.D}, q->options());
    out = &out_new;
  }
  if (want_lse && a[12] == Py_None) {
    lse_new = at::empty({d.T, d.Hq}, q->options().dtype(ScalarType::Float));
    lse = &lse_new;
  }
  const int st = cmp_paged_attention(q->data_ptr(), kc->data_ptr(), vc->data_ptr(), ints(table), ints(cu), start, scale,
                                     window, key_block, key_stride, c.dt, out->data_ptr(),
                                     want_lse ? static_cast<float*>(lse->data_ptr()) : nullptr, ws->data_ptr(), have,
                                     c.stream(), &d);
  if (st != CMP_OK) return status(st);
  if (!want_lse) return THPVariable_Wrap(*out);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyObject* x = THPVariable_Wrap(*out);
  PyObject* y = THPVariable_Wrap(*lse);
  PyTuple_SET_ITEM(r, 0, x);
  PyTuple_SET_ITEM(r, 1, y);
  return r;
}

// C++ exceptions (an allocation that fails, say) become Python's, as torch's own calls raise them.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))guarded<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_norm_rope), FAST(kv_append), FAST(paged_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The package uses the module only with the PyTorch it was built for.
PyMODINIT_FUNC PyInit__fast(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FAST_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
