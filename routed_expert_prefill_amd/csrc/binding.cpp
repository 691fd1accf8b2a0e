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
#include <ATen/EmptyTensor.h>
#include <ATen/detail/CUDAHooksInterface.h>

#include "moe_prefill.h"

namespace {

decltype(&moe_add_rmsnorm) norm_entry = nullptr;
decltype(&moe_decode_ffn) decode_entry = nullptr;
decltype(&moe_route_select) select_entry = nullptr;
decltype(&moe_quant_blocks_fp8) quant_entry = nullptr;
decltype(&moe_matmul_fp8_workspace) matmul_ws_entry = nullptr;
decltype(&moe_matmul_fp8) matmul_entry = nullptr;
decltype(&moe_shared_ffn_workspace) shared_ws_entry = nullptr;
decltype(&moe_shared_ffn) shared_entry = nullptr;

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

// A device and a stream as Python hands them; false where they are not.
bool where(PyObject *device, PyObject *stream, Want *want, void **s) {
  want->device = (int)PyLong_AsLong(device);
  *s = PyLong_AsVoidPtr(stream);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// An int of the C ABI; ok is cleared for anything else.
int32_t whole(PyObject *o, bool *ok) {
  if (!PyLong_CheckExact(o)) {
    *ok = false;
    return 0;
  }
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (over || v < INT32_MIN || v > INT32_MAX) *ok = false;
  return (int32_t)v;
}

// A tensor for outputs or workspace on the device of x, which is the current one.  (The
// allocator's own call: through the dispatcher at::empty takes 0.4 us more.)
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) {
  static c10::Allocator *const allocator = at::detail::getCUDAHooks().getCUDADeviceAllocator();
  return at::detail::empty_generic(sizes, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                   type, std::nullopt);
}

// The result of a call: the given object, or the tensor made for it.
PyObject *result_of(PyObject *given, at::Tensor *made) {
  if (made->defined()) return THPVariable_Wrap(std::move(*made));
  Py_INCREF(given);
  return given;
}
PyObject *pair_of(PyObject *given0, at::Tensor *made0, PyObject *given1, at::Tensor *made1) {
  PyObject *pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyObject *given[2] = {given0, given1};
  at::Tensor *made[2] = {made0, made1};
  for (int i = 0; i < 2; ++i) {
    PyObject *o = result_of(given[i], made[i]);
    if (!o) {
      Py_DECREF(pair);
      return nullptr;
    }
    PyTuple_SET_ITEM(pair, i, o);
  }
  return pair;
}
// The result where the call went well, else what refused() says.
PyObject *finish(PyObject *result, int rc) {
  if (rc == MOE_OK) return result;
  Py_DECREF(result);
  return refused(rc);
}

// route_select(logits, k, scores, bias, groups, top_groups, group_top, renormalise,
// scale, topk_ids, topk_w, device, stream) -> (topk_ids, topk_w), a status or None
PyObject *route_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Want want{0};
  void *stream;
  if (n != 13 || !select_entry || !PyBool_Check(a[7]) || !PyFloat_CheckExact(a[8]) ||
      !where(a[11], a[12], &want, &stream))
    Py_RETURN_NONE;
  bool ok = true;
  moe_select_desc d{};
  d.k = whole(a[1], &ok);
  d.scores = whole(a[2], &ok);
  d.groups = whole(a[4], &ok);
  d.top_groups = whole(a[5], &ok);
  d.group_top = whole(a[6], &ok);
  d.renormalise = a[7] == Py_True;
  d.scale = (float)PyFloat_AS_DOUBLE(a[8]);
  try {
    const at::Tensor *z = want.rows(a[0]);
    if (!ok || !want.ok || z->dim() != 2 || !number(z->scalar_type()) || z->size(0) < 1 ||
        z->size(0) > INT32_MAX || z->size(1) > INT32_MAX || d.k < 1 || d.k > MOE_MAX_TOPK)
      Py_RETURN_NONE;
    d.T = (int32_t)z->size(0);
    d.E = (int32_t)z->size(1);
    d.logits_dtype = dtype(*z);
    const at::Tensor *bias = want.tensor(a[3], {d.E}, at::kFloat, true);
    const at::Tensor *ids = want.tensor(a[9], {d.T, d.k}, at::kInt, true);
    const at::Tensor *w = want.tensor(a[10], {d.T, d.k}, at::kFloat, true);
    if (!want.ok) Py_RETURN_NONE;
    at::Tensor made[2];
    if (!ids) made[0] = fresh({d.T, d.k}, at::kInt), ids = &made[0];
    if (!w) made[1] = fresh({d.T, d.k}, at::kFloat), w = &made[1];
    int32_t *const to_ids = ptr<int32_t>(ids);
    float *const to_w = ptr<float>(w);
    PyObject *result = pair_of(a[9], &made[0], a[10], &made[1]);
    if (!result) return nullptr;
    return finish(result, select_entry(&d, ptr(z), ptr<float>(bias), to_ids, to_w, stream));
  } catch (const std::exception &) {
    Py_RETURN_NONE;
  }
}

// quant_blocks_fp8(x, q, s, device, stream) -> (q, s), a status or None
PyObject *quant_blocks(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Want want{0};
  void *stream;
  if (n != 5 || !quant_entry || !where(a[3], a[4], &want, &stream)) Py_RETURN_NONE;
  try {
    const at::Tensor *x = want.rows(a[0]);
    if (!want.ok || x->dim() != 2 || !number(x->scalar_type()) || x->size(0) < 1 ||
        x->size(0) > INT32_MAX || x->size(1) > INT32_MAX || x->size(1) % 128 != 0)
      Py_RETURN_NONE;
    const int64_t rows = x->size(0), cols = x->size(1);
    const at::Tensor *q = want.tensor(a[1], {rows, cols}, at::kByte, true);
    const at::Tensor *s = want.tensor(a[2], {rows, cols / 128}, at::kFloat, true);
    if (!want.ok) Py_RETURN_NONE;
    at::Tensor made[2];
    if (!q) made[0] = fresh({rows, cols}, at::kByte), q = &made[0];
    if (!s) made[1] = fresh({rows, cols / 128}, at::kFloat), s = &made[1];
    uint8_t *const to_q = ptr<uint8_t>(q);
    float *const to_s = ptr<float>(s);
    PyObject *result = pair_of(a[1], &made[0], a[2], &made[1]);
    if (!result) return nullptr;
    return finish(result, quant_entry(ptr(x), dtype(*x), (int)rows, (int)cols, to_q, to_s, stream));
  } catch (const std::exception &) {
    Py_RETURN_NONE;
  }
}

// Rows of a dense product: bf16, or codes with the scales of their blocks.
struct Rows {
  const at::Tensor *x, *xs;
  int64_t M, K;
};
bool rows_of(Want *want, PyObject *x, PyObject *xs, Rows *r) {
  r->x = want->rows(x);
  if (!want->ok || r->x->dim() != 2 || r->x->size(0) < 1 || r->x->size(0) > INT32_MAX ||
      r->x->size(1) < 1 || r->x->size(1) > INT32_MAX || r->x->size(1) % 128 != 0)
    return false;
  r->M = r->x->size(0);
  r->K = r->x->size(1);
  r->xs = want->tensor(xs, {r->M, r->K / 128}, at::kFloat, true);
  return want->ok && r->x->scalar_type() == (r->xs ? at::kByte : at::kBFloat16);
}

// out as given, or made; the workspace as given, or made with at least `need` bytes.
bool room_of(Want *want, PyObject *given_out, bool f32, int64_t M, int64_t N, const Rows &r,
             PyObject *given_ws, size_t need, at::Tensor *made, const at::Tensor **out,
             at::Tensor *made_ws, const at::Tensor **ws) {
  *out = want->rows(given_out, true);
  *ws = need ? want->rows(given_ws, true) : nullptr;
  if (!want->ok || (*out && (!number((*out)->scalar_type()) ||
                             (*out)->sizes() != at::IntArrayRef({M, N}))) ||
      (*ws && (*ws)->scalar_type() != at::kByte))
    return false;
  if (!*out) {
    *made = fresh({M, N}, f32 ? at::kFloat : at::kBFloat16);
    *out = made;
  }
  if (need && !*ws) {
    *made_ws = fresh({(int64_t)need}, at::kByte);
    *ws = made_ws;
  }
  return true;
}

// matmul_fp8(x, xs, w, s, out, f32, no_type, workspace, device, stream) -> out, a status or None
PyObject *matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Want want{0};
  void *stream;
  if (n != 10 || !matmul_entry || a[6] != Py_False || !where(a[8], a[9], &want, &stream))
    Py_RETURN_NONE;
  try {
    Rows r;
    if (!rows_of(&want, a[0], a[1], &r)) Py_RETURN_NONE;
    const at::Tensor *w = want.rows(a[2]);
    if (!want.ok || w->dim() != 2 || w->scalar_type() != at::kByte || w->size(0) < 1 ||
        w->size(0) > INT32_MAX || w->size(1) != r.K)
      Py_RETURN_NONE;
    const int64_t N = w->size(0);
    const at::Tensor *s = want.tensor(a[3], {(N + 127) / 128, r.K / 128}, at::kFloat);
    if (!want.ok) Py_RETURN_NONE;
    const size_t need = r.xs ? 0 : matmul_ws_entry((int)r.M, (int)N, (int)r.K);
    if (!r.xs && !need) Py_RETURN_NONE;
    at::Tensor made, made_ws;
    const at::Tensor *out, *ws;
    if (!room_of(&want, a[4], a[5] == Py_True, r.M, N, r, a[7], need, &made, &out, &made_ws, &ws))
      Py_RETURN_NONE;
    void *const to = ptr(out);
    const int type = dtype(*out);
    PyObject *result = result_of(a[4], &made);
    if (!result) return nullptr;
    return finish(result, matmul_entry(ptr(r.x), ptr<float>(r.xs), (int)r.M, (int)N, (int)r.K,
                                       ptr<uint8_t>(w), ptr<float>(s), to, type, ptr(ws),
                                       ws ? (size_t)ws->numel() : 0, stream));
  } catch (const std::exception &) {
    Py_RETURN_NONE;
  }
}

// shared_ffn(x, xs, w_gate, w_up, w_down, s_gate, s_up, s_down, out, f32, no_type,
// workspace, device, stream) -> out, a status or None
PyObject *shared_ffn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Want want{0};
  void *stream;
  if (n != 14 || !shared_entry || a[10] != Py_False || !where(a[12], a[13], &want, &stream))
    Py_RETURN_NONE;
  try {
    Rows r;
    if (!rows_of(&want, a[0], a[1], &r)) Py_RETURN_NONE;
    const at::Tensor *wg = want.rows(a[2]);
    if (!want.ok || wg->dim() != 2 || wg->scalar_type() != at::kByte || wg->size(0) < 1 ||
        wg->size(0) > INT32_MAX || wg->size(0) % 128 != 0 || wg->size(1) != r.K)
      Py_RETURN_NONE;
    const int64_t f = wg->size(0), d = r.K;
    const at::Tensor *wu = want.tensor(a[3], {f, d}, at::kByte);
    const at::Tensor *wd = want.tensor(a[4], {d, f}, at::kByte);
    const at::Tensor *sg = want.tensor(a[5], {f / 128, d / 128}, at::kFloat);
    const at::Tensor *su = want.tensor(a[6], {f / 128, d / 128}, at::kFloat);
    const at::Tensor *sd = want.tensor(a[7], {d / 128, f / 128}, at::kFloat);
    if (!want.ok) Py_RETURN_NONE;
    const size_t need = shared_ws_entry((int)r.M, (int)d, (int)f);
    if (!need) Py_RETURN_NONE;
    at::Tensor made, made_ws;
    const at::Tensor *out, *ws;
    if (!room_of(&want, a[8], a[9] == Py_True, r.M, d, r, a[11], need, &made, &out, &made_ws, &ws))
      Py_RETURN_NONE;
    void *const to = ptr(out);
    const int type = dtype(*out);
    PyObject *result = result_of(a[8], &made);
    if (!result) return nullptr;
    return finish(result,
                  shared_entry(ptr(r.x), ptr<float>(r.xs), (int)r.M, (int)d, (int)f,
                               ptr<uint8_t>(wg), ptr<uint8_t>(wu), ptr<uint8_t>(wd), ptr<float>(sg),
                               ptr<float>(su), ptr<float>(sd), to, type, ptr(ws),
                               (size_t)ws->numel(), stream));
  } catch (const std::exception &) {
    Py_RETURN_NONE;
  }
}

// bind_dense(addresses of moe_route_select, moe_quant_blocks_fp8,
// moe_matmul_fp8_workspace, moe_matmul_fp8, moe_shared_ffn_workspace, moe_shared_ffn)
PyObject *bind_dense(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind_dense takes six addresses");
    return nullptr;
  }
  void *p[6];
  for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  select_entry = reinterpret_cast<decltype(select_entry)>(p[0]);
  quant_entry = reinterpret_cast<decltype(quant_entry)>(p[1]);
  matmul_ws_entry = reinterpret_cast<decltype(matmul_ws_entry)>(p[2]);
  matmul_entry = reinterpret_cast<decltype(matmul_entry)>(p[3]);
  shared_ws_entry = reinterpret_cast<decltype(shared_ws_entry)>(p[4]);
  shared_entry = reinterpret_cast<decltype(shared_entry)>(p[5]);
  Py_RETURN_NONE;
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
    {"route_select", reinterpret_cast<PyCFunction>(route_select), METH_FASTCALL, nullptr},
    {"quant_blocks_fp8", reinterpret_cast<PyCFunction>(quant_blocks), METH_FASTCALL, nullptr},
    {"matmul_fp8", reinterpret_cast<PyCFunction>(matmul), METH_FASTCALL, nullptr},
    {"shared_ffn", reinterpret_cast<PyCFunction>(shared_ffn), METH_FASTCALL, nullptr},
    {"bind_dense", reinterpret_cast<PyCFunction>(bind_dense), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
