// Fast path of the Python binding for the paged-cache, sliding-window, tree and
// page entry points: unpacks and checks the tensors of a call in C++ (about 0.3 us instead
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
decltype(&kvcache_append_paged_axes) append_axes = nullptr;
decltype(&kvcache_append_paged_q8_axes) append_q8_axes = nullptr;
decltype(&decode_attn_tree_fwd) tree_fwd = nullptr;
decltype(&decode_attn_tree_q8_fwd) tree_q8_fwd = nullptr;
decltype(&kvcache_resize_paged) resize_paged = nullptr;
decltype(&kvcache_fork_paged) fork_paged = nullptr;
decltype(&kvcache_copy_pages) copy_pages_fn = nullptr;
decltype(&kvcache_compact_paged) compact_paged = nullptr;
decltype(&kvcache_compact_paged_q8) compact_paged_q8 = nullptr;

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
//  q_out, err_flag[, rope_position_ids, rope_axis])
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14 && n != 16) return not_here();
  const bool by_axes = n == 16;
  const Arg turns(by_axes ? a[14] : Py_None, !by_axes), axis(by_axes ? a[15] : Py_None, true);
  if (!turns.ok || !axis.ok) return not_here();
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
  if (by_axes && (!cos || !turns.is(at::kInt, index) || turns->dim() != 2 || turns->size(0) < 1 ||
                  turns->size(0) > DA_MAX_ROPE_AXES || turns->size(1) != tokens || !axis.may_be(at::kInt, index) ||
                  (axis && axis->numel() != D / 2)))
    return not_here();
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
  const int32_t *rows_of = static_cast<const int32_t*>(turns.data()), *axes_of = static_cast<const int32_t*>(axis.data());
  const int axes = by_axes ? (int)turns->size(0) : 0;
  const int status =
      by_axes && eight
          ? append_q8_axes(k.data(), v.data(), static_cast<float*>(ks.data()), static_cast<float*>(vs.data()), k_new.data(),
                           v_new.data(), q.data(), out, c, s, rows, rows_of, axes_of, axes, tab, p, st, (int)B,
                           (int)tokens, H, Hkv, (int)D, pages, size, max_pages, code, e, stream)
      : by_axes
          ? append_axes(k.data(), v.data(), k_new.data(), v_new.data(), q.data(), out, c, s, rows, rows_of, axes_of, axes,
                        tab, p, st, (int)B, (int)tokens, H, Hkv, (int)D, pages, size, max_pages, code, e, stream)
      : eight ? append_paged_q8(k.data(), v.data(), static_cast<float*>(ks.data()), static_cast<float*>(vs.data()),
                              k_new.data(), v_new.data(), q.data(), out, c, s, rows, tab, p, st, (int)B, (int)tokens,
                              H, Hkv, (int)D, pages, size, max_pages, code, e, stream)
            : append_paged(k.data(), v.data(), k_new.data(), v_new.data(), q.data(), out, c, s, rows, tab, p, st,
                           (int)B, (int)tokens, H, Hkv, (int)D, pages, size, max_pages, code, e, stream);
  if (status != DA_OK) return not_here();
  if (!q) Py_RETURN_NONE;
  return q_out ? new_reference(a[12]) : THPVariable_Wrap(std::move(made));
}

// (q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, token_start, tree_mask, out, scale, workspace, err_flag)
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return not_here();
  const Arg q(a[0]), k(a[1]), v(a[2]), ks(a[3], true), vs(a[4], true), table(a[5]), kv_len(a[6]), start(a[7], true),
      mask(a[8], true), out(a[9], true), ws(a[11], true), err(a[12], true);
  if (!(q.ok && k.ok && v.ok && ks.ok && vs.ok && table.ok && kv_len.ok && start.ok && mask.ok && out.ok && ws.ok &&
        err.ok) ||
      !q->is_cuda())
    return not_here();
  const int index = q->get_device(), code = dtype_code(q->scalar_type());
  const bool eight = (bool)ks;
  if (code < 0 || index != c10::cuda::current_device() || q->dim() != 3 || !q.on(index) || !all_fit(q->sizes()) ||
      !pool_ok(k, v, ks, vs, q->scalar_type(), eight, index) || k->size(3) != q->size(2) ||
      !table.is(at::kInt, index) || table->dim() != 2 || !all_fit(table->sizes()) || !kv_len.is(at::kInt, index) ||
      kv_len->numel() != table->size(0) || !start.may_be(at::kInt, index) || !mask.may_be(at::kLong, index))
    return not_here();
  const int64_t B = table->size(0), tokens = q->size(0);
  if (start ? start->numel() != B + 1 : tokens != B) return not_here();
  if (mask && (mask->dim() != 2 || mask->size(0) != tokens || mask->size(1) < 1 ||
               mask->size(1) > DA_TREE_MAX_TOKENS / 64))
    return not_here();
  Tail t;
  if (!t.take(q, out, a[10], ws, err, index)) return not_here();
  const int H = (int)q->size(1), Hkv = (int)k->size(1), D = (int)q->size(2), pages = (int)k->size(0);
  const int size = (int)k->size(2), max_pages = (int)table->size(1), words = mask ? (int)mask->size(1) : 0;
  const int32_t *tab = static_cast<const int32_t*>(table.data()), *len = static_cast<const int32_t*>(kv_len.data()),
                *st = static_cast<const int32_t*>(start.data());
  const int64_t* bits = static_cast<const int64_t*>(mask.data());
  const int status =
      eight ? tree_q8_fwd(q.data(), k.data(), v.data(), static_cast<const float*>(ks.data()),
                          static_cast<const float*>(vs.data()), tab, len, st, bits, words, (int)B, (int)tokens, H, Hkv, D,
                          pages, size, max_pages, t.scale, t.out, t.workspace, t.workspace_bytes, code, t.err, t.stream)
            : tree_fwd(q.data(), k.data(), v.data(), tab, len, st, bits, words, (int)B, (int)tokens, H, Hkv, D, pages, size,
                       max_pages, t.scale, t.out, t.workspace, t.workspace_bytes, code, t.err, t.stream);
  return t.result(a[9], status);
}

// An int32 tensor of one or two dimensions.
bool ints(const Arg& x, int index, int64_t rows, int64_t cols = -1) {
  return x.is(at::kInt, index) && x->dim() == (cols < 0 ? 1 : 2) && x->size(0) == rows && (cols < 0 || x->size(1) == cols);
}

// Pages of a pool's state, or 0.
int pool_pages(const Arg& pool, int index) {
  if (!pool.is(at::kInt, index) || pool->dim() != 1) return 0;
  const int64_t n = pool->numel() - DA_POOL_HEADER;
  return n > 0 && n % 2 == 0 && fits_int(n) ? (int)(n / 2) : 0;
}

bool flag_ok(const Arg& err, int index) { return err.may_be(at::kInt, index) && (!err || err->numel() >= 1); }

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }

// (page_table, held_len, wanted_len, pool, page_size, err_flag)
PyObject* resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return not_here();
  const Arg table(a[0]), held(a[1]), wanted(a[2]), pool(a[3]), err(a[5], true);
  int size;
  if (!(table.ok && held.ok && wanted.ok && pool.ok && err.ok) || !to_int(a[4], &size) || !pool->is_cuda())
    return not_here();
  const int index = pool->get_device(), pages = pool_pages(pool, index);
  if (!pages || index != c10::cuda::current_device() || table->dim() != 2 || !all_fit(table->sizes()) ||
      !table.is(at::kInt, index) || !ints(held, index, table->size(0)) || !ints(wanted, index, table->size(0)) ||
      !flag_ok(err, index))
    return not_here();
  const int status = resize_paged(static_cast<int32_t*>(table.data()), static_cast<const int32_t*>(held.data()),
                                  static_cast<const int32_t*>(wanted.data()), static_cast<int32_t*>(pool.data()),
                                  (int)table->size(0), pages, size, (int)table->size(1),
                                  static_cast<int32_t*>(err.data()), stream_of(index));
  if (status != DA_OK) return not_here();
  Py_RETURN_NONE;
}

// (page_table, kv_len, parent, child, pool, page_size, copies, err_flag)
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) return not_here();
  const Arg table(a[0]), kv_len(a[1]), parent(a[2]), child(a[3]), pool(a[4]), copies(a[6], true), err(a[7], true);
  int size;
  if (!(table.ok && kv_len.ok && parent.ok && child.ok && pool.ok && copies.ok && err.ok) || !to_int(a[5], &size) ||
      !pool->is_cuda())
    return not_here();
  const int index = pool->get_device(), pages = pool_pages(pool, index);
  const int64_t forks = parent->numel();
  if (!pages || index != c10::cuda::current_device() || table->dim() != 2 || !all_fit(table->sizes()) ||
      !table.is(at::kInt, index) || !ints(kv_len, index, table->size(0)) || !fits_int(forks) ||
      !ints(parent, index, forks) || !ints(child, index, forks) || (copies && !ints(copies, index, 3, forks)) ||
      !flag_ok(err, index))
    return not_here();
  at::Tensor made;
  if (!copies) made = at::empty({3, forks}, pool->options());
  const int status = fork_paged(static_cast<int32_t*>(table.data()), static_cast<int32_t*>(kv_len.data()),
                                static_cast<const int32_t*>(parent.data()), static_cast<const int32_t*>(child.data()),
                                static_cast<int32_t*>(pool.data()),
                                static_cast<int32_t*>(copies ? copies.data() : made.data_ptr()), (int)forks,
                                (int)table->size(0), pages, size, (int)table->size(1),
                                static_cast<int32_t*>(err.data()), stream_of(index));
  if (status != DA_OK) return not_here();
  return copies ? new_reference(a[6]) : THPVariable_Wrap(std::move(made));
}

// Pools of one layer or of several, and their scales (or none).
struct Stack {
  int index, layers, pages, heads, size, head_dim, element;

  bool take(const Arg& k, const Arg& v, const Arg& ks, const Arg& vs) {
    if (!k->is_cuda()) return false;
    index = k->get_device();
    const at::ScalarType type = k->scalar_type();
    const bool eight = type == at::kFloat8_e4m3fn;
    if (index != c10::cuda::current_device() || (dtype_code(type) < 0 && !eight) || (k->dim() != 4 && k->dim() != 5) ||
        v->sizes() != k->sizes() || !k.is(type, index) || !v.is(type, index) || !all_fit(k->sizes()) ||
        (bool)ks != (bool)vs || (ks && !eight))
      return false;
    if (ks && (ks->sizes() != k->sizes().slice(0, k->dim() - 2) || vs->sizes() != ks->sizes() ||
               !ks.is(at::kFloat, index) || !vs.is(at::kFloat, index)))
      return false;
    const int lead = (int)k->dim() - 4;
    layers = lead ? (int)k->size(0) : 1;
    pages = (int)k->size(lead);
    heads = (int)k->size(lead + 1);
    size = (int)k->size(lead + 2);
    head_dim = (int)k->size(lead + 3);
    element = eight ? 1 : 2;
    return true;
  }
};

// (k_pages, v_pages, k_scale, v_scale, copies, err_flag)
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return not_here();
  const Arg k(a[0]), v(a[1]), ks(a[2], true), vs(a[3], true), copies(a[4]), err(a[5], true);
  Stack s;
  if (!(k.ok && v.ok && ks.ok && vs.ok && copies.ok && err.ok) || !s.take(k, v, ks, vs) || copies->dim() != 2 ||
      !fits_int(copies->size(1)) || !ints(copies, s.index, 3, copies->size(1)) || !flag_ok(err, s.index))
    return not_here();
  const int status = copy_pages_fn(k.data(), v.data(), static_cast<float*>(ks.data()), static_cast<float*>(vs.data()),
                                   static_cast<const int32_t*>(copies.data()), (int)copies->size(1), s.layers, s.pages,
                                   s.heads, s.size, s.head_dim, s.element, static_cast<int32_t*>(err.data()),
                                   stream_of(s.index));
  if (status != DA_OK) return not_here();
  Py_RETURN_NONE;
}

// (k_pages, v_pages, k_scale, v_scale, page_table, keep, keep_start, position_ids, err_flag)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return not_here();
  const Arg k(a[0]), v(a[1]), ks(a[2], true), vs(a[3], true), table(a[4]), keep(a[5]), start(a[6]), pos(a[7]),
      err(a[8], true);
  Stack s;
  if (!(k.ok && v.ok && ks.ok && vs.ok && table.ok && keep.ok && start.ok && pos.ok && err.ok) || !s.take(k, v, ks, vs) ||
      (s.element == 1) != (bool)ks || table->dim() != 2 || !all_fit(table->sizes()) || !table.is(at::kInt, s.index) ||
      !fits_int(keep->numel()) || !ints(keep, s.index, keep->numel()) || !ints(start, s.index, table->size(0) + 1) ||
      !ints(pos, s.index, table->size(0)) || !flag_ok(err, s.index))
    return not_here();
  const int32_t *tab = static_cast<const int32_t*>(table.data()), *rows = static_cast<const int32_t*>(keep.data()),
                *st = static_cast<const int32_t*>(start.data()), *p = static_cast<const int32_t*>(pos.data());
  int32_t* const e = static_cast<int32_t*>(err.data());
  const int B = (int)table->size(0), kept = (int)keep->numel(), most = (int)table->size(1);
  const int status =
      ks ? compact_paged_q8(k.data(), v.data(), static_cast<float*>(ks.data()), static_cast<float*>(vs.data()), tab, rows,
                            st, p, B, kept, s.layers, s.heads, s.head_dim, s.pages, s.size, most, e, stream_of(s.index))
         : compact_paged(k.data(), v.data(), tab, rows, st, p, B, kept, s.layers, s.heads, s.head_dim, s.pages, s.size,
                         most, e, stream_of(s.index));
  if (status != DA_OK) return not_here();
  Py_RETURN_NONE;
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

// bind(addresses of the entry points, in the order of the declarations above)
PyObject* bind(PyObject*, PyObject* args) {
  constexpr int kCount = 14;
  void* f[kCount];
  if (!PyTuple_Check(args) || PyTuple_GET_SIZE(args) != kCount) {
    PyErr_SetString(PyExc_TypeError, "bind takes the addresses of every entry point");
    return nullptr;
  }
  for (int i = 0; i < kCount; ++i) {
    f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, i));
    if (PyErr_Occurred()) return nullptr;
  }
  paged_fwd = reinterpret_cast<decltype(paged_fwd)>(f[0]);
  paged_q8_fwd = reinterpret_cast<decltype(paged_q8_fwd)>(f[1]);
  window_fwd = reinterpret_cast<decltype(window_fwd)>(f[2]);
  append_paged = reinterpret_cast<decltype(append_paged)>(f[3]);
  append_paged_q8 = reinterpret_cast<decltype(append_paged_q8)>(f[4]);
  append_axes = reinterpret_cast<decltype(append_axes)>(f[5]);
  append_q8_axes = reinterpret_cast<decltype(append_q8_axes)>(f[6]);
  tree_fwd = reinterpret_cast<decltype(tree_fwd)>(f[7]);
  tree_q8_fwd = reinterpret_cast<decltype(tree_q8_fwd)>(f[8]);
  resize_paged = reinterpret_cast<decltype(resize_paged)>(f[9]);
  fork_paged = reinterpret_cast<decltype(fork_paged)>(f[10]);
  copy_pages_fn = reinterpret_cast<decltype(copy_pages_fn)>(f[11]);
  compact_paged = reinterpret_cast<decltype(compact_paged)>(f[12]);
  compact_paged_q8 = reinterpret_cast<decltype(compact_paged_q8)>(f[13]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<attn_paged>("attn_paged"), method<attn_window>("attn_window"),
                         method<append>("append"),
                         method<attn_tree>("attn_tree"),
                         method<resize>("resize"),
                         method<fork>("fork"),
                         method<copy_pages>("copy_pages"),
                         method<compact>("compact"),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
