// Fast path of the Python binding for the paged-cache and sliding-window entry
// points: unpacks and checks the tensors of a call in C++ (about 0.3 us instead
// of 5 us of attribute look-ups in Python) and makes it. A call whose arguments
// are not all as documented, or that the library refuses, returns
// NotImplemented and is left to the Python path, which says what is wrong.
#include <ATen/ATen.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "decode_attn.h"

namespace {

decltype(&decode_attn_paged_fwd) paged_fwd = nullptr;
decltype(&decode_attn_paged_q8_fwd) paged_q8_fwd = nullptr;
decltype(&decode_attn_window_fwd) window_fwd = nullptr;
decltype(&kvcache_append_paged) append_paged = nullptr;
decltype(&kvcache_append_paged_q8) append_paged_q8 = nullptr;

// A tensor argument, or null where None is allowed and given.
struct Arg {
  const at::Tensor* t = nullptr;
  bool ok = true;

  Arg(PyObject* o, bool optional = false) {
    if (optional && o == Py_None) return;
    if (THPVariable_Check(o)) {
      t = &THPVariable_Unpack(o);
    } else {
      ok = false;
    }
  }
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor* operator->() const { return t; }
  void* data() const { return t ? t->data_ptr() : nullptr; }
  // A dense tensor of this type on device `index`.
  bool is(at::ScalarType type, int index) const {
    return t->scalar_type() == type && on(index);
  }
  bool on(int index) const {
    return t->is_cuda() && t->get_device() == index && t->is_contiguous();
  }
  // As is(), or not given.
  bool may_be(at::ScalarType type, int index) const { return !t || is(type, index); }
};

bool fits_int(int64_t n) { return n >= 0 && n <= INT32_MAX; }

bool all_fit(at::IntArrayRef sizes) {
  for (const int64_t n : sizes)
    if (!fits_int(n)) return false;
  return true;
}

// The library's code of a query type, or -1.
int dtype_code(at::ScalarType t) { return t == at::kHalf ? DA_F16 : t == at::kBFloat16 ? DA_BF16 : -1; }

bool to_int(PyObject* o, int* out) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (overflow || v < INT32_MIN || v > INT32_MAX) return false;
  *out = (int)v;
  return true;
}

bool to_scale(PyObject* o, int64_t head_dim, float* out) {
  if (o == Py_None) {
    *out = (float)(1.0 / std::sqrt((double)head_dim));
    return true;
  }
  if (!PyFloat_CheckExact(o)) return false;
  *out = (float)PyFloat_AS_DOUBLE(o);
  return true;
}

PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }

PyObject* new_reference(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// Pools of a paged cache: shapes and types of pages and scales.
bool pool_ok(const Arg& k, const Arg& v, const Arg& ks, const Arg& vs, at::ScalarType dtype, bool eight, int index) {
  const at::ScalarType store = eight ? at::kFloat8_e4m3fn : dtype;
  if (k->dim() != 4 || v->sizes() != k->sizes() || !k.is(store, index) || !v.is(store, index) || !all_fit(k->sizes()))
    return false;
  if (!eight) return true;
  return ks && vs && ks->sizes() == k->sizes().slice(0, 2) && vs->sizes() == ks->sizes() && ks.is(at::kFloat, index) &&
         vs.is(at::kFloat, index);
}

// The arguments that every attention call ends with.
struct Tail {
  at::Tensor made;  // the output, where none was given
  void* out;
  float scale;
  void* workspace;
  size_t workspace_bytes;
  int32_t* err;
  void* stream;

  bool take(const Arg& q, const Arg& given, PyObject* scale_arg, const Arg& ws, const Arg& err_flag, int index) {
    if (!ws || !ws.on(index) || !err_flag.may_be(at::kInt, index) || (err_flag && err_flag->numel() < 1)) return false;
    if (given && (given->sizes() != q->sizes() || !given.is(q->scalar_type(), index))) return false;
    if (!to_scale(scale_arg, q->size(2), &scale)) return false;
    if (!given) made = at::empty_like(*q.t);
    out = given ? given.data() : made.data_ptr();
    workspace = ws.data();
    workspace_bytes = ws->nbytes();
    err = static_cast<int32_t*>(err_flag.data());
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    return true;
  }
  PyObject* result(PyObject* given, int status) {
    if (status != DA_OK) return not_here();
    return given == Py_None ? THPVariable_Wrap(std::move(made)) : new_reference(given);
  }
};

// (q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, window, sinks, out, scale, workspace, err_flag)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return not_here();
  const Arg q(a[0]), k(a[1]), v(a[2]), ks(a[3], true), vs(a[4], true), table(a[5]), kv_len(a[6]), out(a[9], true),
      ws(a[11], true), err(a[12], true);
  int window, sinks;
  if (!(q.ok && k.ok && v.ok && ks.ok && vs.ok && table.ok && kv_len.ok && out.ok && ws.ok && err.ok) ||
      !to_int(a[7], &window) || !to_int(a[8], &sinks) || !q->is_cuda())
    return not_here();
  const int index = q->get_device(), code = dtype_code(q->scalar_type());
  const bool eight = (bool)ks;
  if (code < 0 || index != c10::cuda::current_device() || q->dim() != 3 || !q.on(index) || !all_fit(q->sizes()) ||
      !pool_ok(k, v, ks, vs, q->scalar_type(), eight, index) || k->size(3) != q->size(2) ||
      !table.is(at::kInt, index) || table->dim() != 2 || table->size(0) != q->size(0) || !all_fit(table->sizes()) ||
      !kv_len.is(at::kInt, index) || kv_len->numel() != q->size(0))
    return not_here();
  Tail t;
  if (!t.take(q, out, a[10], ws, err, index)) return not_here();
  const int B = (int)q->size(0), H = (int)q->size(1), Hkv = (int)k->size(1), D = (int)q->size(2);
  const int pages = (int)k->size(0), size = (int)k->size(2), max_pages = (int)table->size(1);
  const int32_t* tab = static_cast<const int32_t*>(table.data());
  const int32_t* len = static_cast<const int32_t*>(kv_len.data());
  const int status =
      eight ? paged_q8_fwd(q.data(), k.data(), v.data(), static_cast<const float*>(ks.data()),
                           static_cast<const float*>(vs.data()), tab, len, B, H, Hkv, D, pages, size, max_pages, window,
                           sinks, t.scale, t.out, t.workspace, t.workspace_bytes, code, t.err, t.stream)
            : paged_fwd(q.data(), k.data(), v.data(), tab, len, B, H, Hkv, D, pages, size, max_pages, window, sinks,
                        t.scale, t.out, t.workspace, t.workspace_bytes, code, t.err, t.stream);
  return t.result(a[9], status);
}

// (q, k_cache, v_cache, kv_len, window, sinks, out, scale, workspace, err_flag)
PyObject* attn_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) return not_here();
  const Arg q(a[0]), k(a[1]), v(a[2]), kv_len(a[3]), out(a[6], true), ws(a[8], true), err(a[9], true);
  int window, sinks;
  if (!(q.ok && k.ok && v.ok && kv_len.ok && out.ok && ws.ok && err.ok) || !to_int(a[4], &window) ||
      !to_int(a[5], &sinks) || !q->is_cuda())
    return not_here();
  const int index = q->get_device(), code = dtype_code(q->scalar_type());
  if (code < 0 || index != c10::cuda::current_device() || q->dim() != 3 || !q.on(index) || !all_fit(q->sizes()) ||
      k->dim() != 4 || v->sizes() != k->sizes() || !k.is(q->scalar_type(), index) || !v.is(q->scalar_type(), index) ||
      !all_fit(k->sizes()) || k->size(0) != q->size(0) || k->size(3) != q->size(2) || !kv_len.is(at::kInt, index) ||
      kv_len->numel() != q->size(0))
    return not_here();
  Tail t;
  if (!t.take(q, out, a[7], ws, err, index)) return not_here();
  const int status = window_fwd(q.data(), k.data(), v.data(), static_cast<const int32_t*>(kv_len.data()),
                                (int)q->size(0), (int)q->size(1), (int)k->size(1), (int)q->size(2), (int)k->size(2),
                                window, sinks, t.scale, t.out, t.workspace, t.workspace_bytes, code, t.err, t.stream);
  return t.result(a[6], status);
}

// (k_pages, v_pages, k_scale, v_scale, k_new, v_new, page_table, position_ids, token_start, rope_cos, rope_sin, q,
//  q_out, err_flag)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) return not_here();
  const Arg k(a[0]), v(a[1]), ks(a[2], true), vs(a[3], true), k_new(a[4]), v_new(a[5]), table(a[6]), pos(a[7]),
      start(a[8], true), cos(a[9], true), sin(a[10], true), q(a[11], true), q_out(a[12], true), err(a[13], true);
  if (!(k.ok && v.ok && ks.ok && vs.ok && k_new.ok && v_new.ok && table.ok && pos.ok && start.ok && cos.ok && sin.ok &&
        q.ok && q_out.ok && err.ok) ||
      !k_new->is_cuda())
    return not_here();
  const at::ScalarType dtype = k_new->scalar_type();
  const int index = k_new->get_device(), code = dtype_code(dtype);
  const bool eight = (bool)ks;
  if (code < 0 || index != c10::cuda::current_device() || k_new->dim() != 3 || !k_new.on(index) ||
      !all_fit(k_new->sizes()) || v_new->sizes() != k_new->sizes() || !v_new.is(dtype, index) ||
      !pool_ok(k, v, ks, vs, dtype, eight, index) || k_new->size(1) != k->size(1) || k_new->size(2) != k->size(3) ||
      !table.is(at::kInt, index) || table->dim() != 2 || !all_fit(table->sizes()) || !pos.is(at::kInt, index) ||
      pos->numel() != table->size(0) || !start.may_be(at::kInt, index) || !err.may_be(at::kInt, index) ||
      (err && err->numel() < 1))
    return not_here();
  const int64_t tokens = k_new->size(0), B = table->size(0), D = k_new->size(2);
  if (start ? start->numel() != B + 1 : tokens != B) return not_here();
  if ((bool)cos != (bool)sin || !cos.may_be(at::kFloat, index) || !sin.may_be(at::kFloat, index)) return not_here();
  if (cos && (cos->dim() != 2 || cos->size(1) != D || sin->sizes() != cos->sizes() || !all_fit(cos->sizes())))
    return not_here();
  if (q ? !cos || q->dim() != 3 || q->size(0) != tokens || q->size(2) != D || !q.is(dtype, index) ||
              !all_fit(q->sizes())
        : (bool)q_out)
    return not_here();
  if (q_out && (q_out->sizes() != q->sizes() || !q_out.is(dtype, index))) return not_here();
  at::Tensor made;
  if (q && !q_out) made = at::empty_like(*q.t);
  void* const out = q ? (q_out ? q_out.data() : made.data_ptr()) : nullptr;
  void* const stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  const float *c = static_cast<const float*>(cos.data()), *s = static_cast<const float*>(sin.data());
  const int32_t *tab = static_cast<const int32_t*>(table.data()), *p = static_cast<const int32_t*>(pos.data()),
                *st = static_cast<const int32_t*>(start.data());
  int32_t* const e = static_cast<int32_t*>(err.data());
  const int rows = cos ? (int)cos->size(0) : 0, H = q ? (int)q->size(1) : 0, Hkv = (int)k->size(1);
  const int pages = (int)k->size(0), size = (int)k->size(2), max_pages = (int)table->size(1);
  const int status =
      eight ? append_paged_q8(k.data(), v.data(), static_cast<float*>(ks.data()), static_cast<float*>(vs.data()),
                              k_new.data(), v_new.data(), q.data(), out, c, s, rows, tab, p, st, (int)B, (int)tokens,
                              H, Hkv, (int)D, pages, size, max_pages, code, e, stream)
            : append_paged(k.data(), v.data(), k_new.data(), v_new.data(), q.data(), out, c, s, rows, tab, p, st,
                           (int)B, (int)tokens, H, Hkv, (int)D, pages, size, max_pages, code, e, stream);
  if (status != DA_OK) return not_here();
  if (!q) Py_RETURN_NONE;
  return q_out ? new_reference(a[12]) : THPVariable_Wrap(std::move(made));
}

// Exceptions of torch become NotImplemented as well: the Python path meets them again.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception&) {
    return not_here();
  }
}

// bind(addresses of the five entry points, in the order of the declarations above)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "KKKKK", f, f + 1, f + 2, f + 3, f + 4)) return nullptr;
  paged_fwd = reinterpret_cast<decltype(paged_fwd)>(f[0]);
  paged_q8_fwd = reinterpret_cast<decltype(paged_q8_fwd)>(f[1]);
  window_fwd = reinterpret_cast<decltype(window_fwd)>(f[2]);
  append_paged = reinterpret_cast<decltype(append_paged)>(f[3]);
  append_paged_q8 = reinterpret_cast<decltype(append_paged_q8)>(f[4]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<attn_paged>("attn_paged"), method<attn_window>("attn_window"),
                         method<append>("append"),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
