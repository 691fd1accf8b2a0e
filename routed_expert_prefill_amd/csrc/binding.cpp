// The Python calls whose kernels take a few microseconds, from tensors to the
// C ABI without the interpreter: the checks of arguments, the outputs'
// allocation and the call.  From Python the same takes 10 to 14 us a call (a
// dozen tensors' types, shapes, devices and strides, a ctypes call of up to 17
// arguments), more than one token's kernels.
//
// Each function returns None for whatever is not a plain good call -- another
// type, shape or device, a status of the argument checks -- and the Python
// code then checks and calls by itself, so that every refusal has one place and
// one wording.  A status of the launch itself is returned as it is, for Python
// to raise: the kernel may have run, and an addition in place must not run
// again.  For the same reason nothing that can fail follows the call.
// The library is not linked: bind() takes the entry points of the one loaded.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include "moe_prefill.h"

namespace {

decltype(&moe_add_rmsnorm) norm_entry = nullptr;
decltype(&moe_decode_ffn) decode_entry = nullptr;

// What a tensor has to be.
struct Want {
  int device;
  bool ok = true;

  // The tensor in o, checked; NULL (and ok) for None where that is allowed.
  const at::Tensor *tensor(PyObject *o, at::IntArrayRef sizes, at::ScalarType type,
                           bool optional = false) {
    const at::Tensor *t = rows(o, optional);
    if (t && ok) ok = t->scalar_type() == type && t->sizes() == sizes;
    return t;
  }
  // The same without its type and sizes.
  const at::Tensor *rows(PyObject *o, bool optional = false) {
    if (!ok || (optional && o == Py_None)) return nullptr;
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    ok = t.layout() == at::kStrided && t.device().type() == at::kCUDA &&
         t.device().index() == device && t.is_contiguous();
    return &t;
  }
};

template <typename T = void>
T *ptr(const at::Tensor *t) {
  return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

// What a function returns for a status other than MOE_OK.
PyObject *refused(int status) {
  if (status == MOE_EHIP) return PyLong_FromLong(status);
  Py_RETURN_NONE;
}

bool number(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
int dtype(const at::Tensor &t) { return t.scalar_type() == at::kFloat ? MOE_DT_F32 : MOE_DT_BF16; }

// add_rmsnorm(x, weight, eps, residual, residual_out, y, q, s, want_bf16,
// want_fp8, device, stream) -> (y, residual_out, q, s), a status or None
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 12 || !norm_entry || !PyBool_Check(a[8]) || !PyBool_Check(a[9])) Py_RETURN_NONE;
  Want want{(int)PyLong_AsLong(a[10])};
  const double eps = PyFloat_AsDouble(a[2]);
  void *stream = PyLong_AsVoidPtr(a[11]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  try {
    const at::Tensor *x = want.rows(a[0]), *w = want.rows(a[1]), *r = want.rows(a[3], true);
    if (!want.ok || x->dim() != 2 || !number(x->scalar_type()) || !number(w->scalar_type()) ||
        w->dim() != 1 || w->size(0) != x->size(1) || x->size(0) < 1 ||
        x->size(0) > INT32_MAX || x->size(1) > INT32_MAX)
      Py_RETURN_NONE;
    if (r && (!number(r->scalar_type()) || r->sizes() != x->sizes())) Py_RETURN_NONE;
    const at::Tensor &like = r ? *r : *x;
    const int64_t rows = x->size(0);
    const at::Tensor *ro = want.tensor(a[4], x->sizes(), like.scalar_type(), true);
    const at::Tensor *y = want.tensor(a[5], x->sizes(), at::kBFloat16, true);
    const at::Tensor *q = want.tensor(a[6], x->sizes(), at::kByte, true);
    const at::Tensor *s = want.tensor(a[7], {rows}, at::kFloat, true);
    if (!want.ok) Py_RETURN_NONE;
    at::Tensor made[4];  // y, residual_out, q, s
    if (!y && a[8] == Py_True) made[0] = at::empty_like(*x, x->options().dtype(at::kBFloat16));
    if (!ro && r) made[1] = at::empty_like(*r);
    if (!q && (a[9] == Py_True || s)) made[2] = at::empty_like(*x, x->options().dtype(at::kByte));
    if (!s && (q || made[2].defined())) made[3] = at::empty({rows}, x->options().dtype(at::kFloat));
    const at::Tensor *out[4] = {y, ro, q, s};
    static const int given[4] = {5, 4, 6, 7};
    for (int i = 0; i < 4; ++i)
      if (!out[i] && made[i].defined()) out[i] = &made[i];
    void *to[4];
    for (int i = 0; i < 4; ++i) to[i] = ptr(out[i]);
    PyObject *result = PyTuple_New(4);
    if (!result) return nullptr;
    for (int i = 0; i < 4; ++i) {
      PyObject *o = made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : a[given[i]];
      if (!o) {
        Py_DECREF(result);
        return nullptr;
      }
      if (o == a[given[i]]) Py_INCREF(o);
      PyTuple_SET_ITEM(result, i, o);
    }
    const int rc = norm_entry(ptr(x), dtype(*x), ptr(r), to[1], dtype(like), ptr(w), dtype(*w),
                              (float)eps, (int)rows, (int)x->size(1), to[0],
                              static_cast<uint8_t *>(to[2]), static_cast<float *>(to[3]), stream);
    if (rc == MOE_OK) return result;
    Py_DECREF(result);
    return refused(rc);
  } catch (const std::exception &) {
    Py_RETURN_NONE;
  }
}

// decode_ffn(x, topk_ids, topk_w, route_mask, w_gate, w_up, w_down, s_gate,
// s_up, s_down, shared, out, workspace, device, stream) -> True, a status or None
PyObject *decode_ffn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 15 || !decode_entry) Py_RETURN_NONE;
  Want want{(int)PyLong_AsLong(a[13])};
  void *stream = PyLong_AsVoidPtr(a[14]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  try {
    const at::Tensor *x = want.rows(a[0]), *ids = want.rows(a[1]), *wg = want.rows(a[4]);
    if (!want.ok || x->dim() != 2 || ids->dim() != 2 || wg->dim() != 3 ||
        x->scalar_type() != at::kBFloat16 || ids->scalar_type() != at::kInt)
      Py_RETURN_NONE;
    const int64_t T = x->size(0), d = x->size(1), k = ids->size(1), E = wg->size(0),
                  f = wg->size(1);
    if (ids->size(0) != T || T < 1 || T > INT16_MAX || k > INT16_MAX || E > INT16_MAX ||
        d > INT32_MAX || f > INT32_MAX)
      Py_RETURN_NONE;
    const at::Tensor *w = want.tensor(a[2], {T, k}, at::kFloat);
    const at::Tensor *mask = want.tensor(a[3], {T, k}, at::kByte, true);
    want.tensor(a[4], {E, f, d / 2}, at::kByte);
    const at::Tensor *wu = want.tensor(a[5], {E, f, d / 2}, at::kByte);
    const at::Tensor *wd = want.tensor(a[6], {E, d, f / 2}, at::kByte);
    const at::Tensor *sg = want.tensor(a[7], {E, f, d / 32}, at::kByte);
    const at::Tensor *su = want.tensor(a[8], {E, f, d / 32}, at::kByte);
    const at::Tensor *sd = want.tensor(a[9], {E, d, f / 32}, at::kByte);
    const at::Tensor *shared = want.tensor(a[10], {T, d}, at::kFloat, true);
    const at::Tensor *out = want.rows(a[11]), *ws = want.rows(a[12]);
    if (!want.ok || !number(out->scalar_type()) || out->sizes() != at::IntArrayRef({T, d}) ||
        ws->scalar_type() != at::kByte)
      Py_RETURN_NONE;
    const bool f32 = out->scalar_type() == at::kFloat;
    const moe_ffn_desc desc = {(int32_t)T, (int32_t)k, (int32_t)E, (int32_t)d, (int32_t)f,
                               MOE_W_MXFP4, MOE_ACT_BF16};
    const int rc = decode_entry(
        &desc, ptr(x), ptr<int32_t>(ids), ptr<float>(w), ptr<uint8_t>(mask), ptr(wg), ptr(wu),
        ptr(wd), ptr(sg), ptr(su), ptr(sd), ptr<float>(shared), f32 ? ptr<float>(out) : nullptr,
        f32 ? nullptr : ptr(out), ptr(ws), (size_t)ws->numel(), stream);
    if (rc != MOE_OK) return refused(rc);
    Py_RETURN_TRUE;
  } catch (const std::exception &) {
    Py_RETURN_NONE;
  }
}

// bind(address of moe_add_rmsnorm, address of moe_decode_ffn)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "bind takes two addresses");
    return nullptr;
  }
  void *norm = PyLong_AsVoidPtr(a[0]), *decode = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return nullptr;
  norm_entry = reinterpret_cast<decltype(norm_entry)>(norm);
  decode_entry = reinterpret_cast<decltype(decode_entry)>(decode);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"add_rmsnorm", reinterpret_cast<PyCFunction>(add_rmsnorm), METH_FASTCALL, nullptr},
    {"decode_ffn", reinterpret_cast<PyCFunction>(decode_ffn), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
