// paged_binding.cpp - the Python binding of the paged operators (page plan,
// rotation, norm of query and key heads, paged K/V decode): checks of torch
// tensors, their outputs and workspaces, and one call of the C ABI. A step of a
// serving loop makes several of these calls, each a few microseconds of GPU
// time; marshalling them in interpreted Python took longer than that (per call,
// launch included, against here: rotation 11.5 / 5.4 us, norm + rotation into
// pages 16 / 6.3, its gradient 27.5 / 11.4, page plan 15.5 / 8.8, decode 21 /
// 8.9), so this part of the binding is compiled. No arithmetic on data happens
// here, and nothing is kept between calls but the addresses of the C functions,
// which paged.py hands over.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <initializer_list>
#include <string>

#include "loza_ssa.h"

namespace {

decltype(&loza_page_plan) f_page_plan;
decltype(&loza_rope) f_rope;
decltype(&loza_qk_norm_rope) f_norm_rope;
decltype(&loza_qk_norm_rope_backward) f_norm_rope_backward;
decltype(&loza_qk_norm_rope_workspace_size) f_norm_rope_workspace;
decltype(&loza_ssa_decode_paged_kv) f_decode;
decltype(&loza_decode_paged_kv_workspace_size) f_decode_workspace;
PyObject* g_status_error;  // LozaError(status, what)
PyObject* g_memory_error;  // torch.OutOfMemoryError
PyObject *g_rope_params, *g_window_params;  // the classes RopeParams and Params

// What a call cannot take: raised as TypeError or ValueError; a status of the C ABI as LozaError.
struct Refused {
  PyObject* type;
  std::string what;
};
struct Status {
  int code;
  const char* what;
};
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
struct PythonError {};  // already set

bool none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
int32_t int32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}

// RopeParams and Params are ctypes structures laid out like the C ones, of the same size: their class tells them apart.
template <typename T>
T params(PyObject* o, PyObject* type, const char* what) {
  const int is = PyObject_IsInstance(o, type);
  if (is < 0) throw PythonError{};
  if (!is) type_error(what);
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw PythonError{};
  T v;
  const bool fits = b.len == (Py_ssize_t)sizeof(T);
  if (fits) memcpy(&v, b.buf, sizeof(T));
  PyBuffer_Release(&b);
  if (!fits) type_error(what);
  return v;
}
loza_rope_params rope_params(PyObject* o) {
  return params<loza_rope_params>(o, g_rope_params, "rope must be a RopeParams");
}

// A call's device, from its first tensor; made current for the call.
struct Place {
  at::Device device;
  c10::cuda::CUDAGuard guard;
  explicit Place(const at::Tensor& first, const char* name) : device(on_gpu(first, name)), guard(device) {}
  static at::Device on_gpu(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    return t.device();
  }
  loza_stream_t stream() const {
    return reinterpret_cast<loza_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype) const {
    return at::empty(sizes, at::TensorOptions().dtype(dtype).device(device));
  }
};

void typed(const at::Tensor& t, const char* name, const Place& at, at::ScalarType dtype) {
  if (t.device() != at.device) {
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    value_error(std::string(name) + " must be on the first tensor's device");
  }
  if (t.scalar_type() != dtype) type_error(std::string(name) + " must be " + c10::toString(dtype));
}
void shaped(const at::Tensor& t, const char* name, at::IntArrayRef sizes) {
  if (t.sizes() == sizes) return;
  std::string s = std::string(name) + " must have shape (";
  for (int64_t n : sizes) s += std::to_string(n) + ", ";
  value_error(s + ")");
}

// Address of a contiguous tensor of exactly this type and shape.
void* plain(PyObject* o, const char* name, const Place& at, at::ScalarType dtype, at::IntArrayRef sizes) {
  const at::Tensor& t = tensor(o, name);
  typed(t, name, at, dtype);
  shaped(t, name, sizes);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// [rows, heads, dim] with heads and dim contiguous within a row.
struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
  Rows() = default;
  Rows(const at::Tensor& t, const char* name, const Place& at, at::ScalarType dtype, at::IntArrayRef sizes) {
    typed(t, name, at, dtype);
    shaped(t, name, sizes);
    const auto s = t.strides();
    if ((s[2] != 1 && sizes[2] > 1) || (s[1] != sizes[2] && sizes[1] > 1))
      value_error(std::string(name) + ": heads and head dim must be contiguous within a row");
    p = t.data_ptr();
    stride = sizes[0] > 1 ? s[0] : sizes[1] * sizes[2];  // of one row: any that fits
  }
};
const at::Tensor& rank(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims) value_error(std::string(name) + " must have " + std::to_string(dims) + " dimensions");
  return t;
}

// A tensor that a call has written in place: autograd then notices that what it had saved of it is gone. (Tensors of
// inference mode keep no count.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// An output: the caller's (checked) or a new one; `made` keeps a new one until it is wrapped.
struct Output {
  PyObject* given = nullptr;
  at::Tensor made;
  PyObject* take() {
    if (given) {
      written(THPVariable_Unpack(given));
      return Py_NewRef(given);
    }
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(Py_None);
  }
};
Rows rows_out(Output* out, PyObject* o, const char* name, const Place& at, at::ScalarType dtype,
              at::IntArrayRef sizes) {
  if (!none(o)) {
    out->given = o;
    return Rows(tensor(o, name), name, at, dtype, sizes);
  }
  out->made = at.empty(sizes, dtype);
  Rows r;
  r.p = out->made.data_ptr();
  r.stride = sizes[1] * sizes[2];
  return r;
}

int dtype_code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return LOZA_BF16;
    case at::kHalf: return LOZA_FP16;
    case at::kFloat: return LOZA_FP32;
    default: type_error(std::string(name) + " must be bfloat16, float16 or float32");
  }
}

// A block table [batch, columns] with contiguous rows.
struct Table {
  int32_t* p;
  int64_t stride, cols;
  Table(PyObject* o, const Place& at, int64_t batch) {
    const at::Tensor& t = rank(o, "block_table", 2);
    typed(t, "block_table", at, at::kInt);
    cols = t.size(1);
    if (t.size(0) != batch || (t.stride(1) != 1 && cols > 1))
      value_error("block_table must be [batch, columns] with contiguous rows");
    p = t.data_ptr<int32_t>();
    stride = batch > 1 ? t.stride(0) : cols;
  }
};

// One of a cache's pools [pages, rows, heads, dim], into `pool`.
void pool_side(loza_kv_pool* pool, bool values, PyObject* o, const Place& at, at::ScalarType dtype, int64_t heads,
               int64_t dim) {
  const char* name = values ? "v_pool" : "k_pool";
  const at::Tensor& t = rank(o, name, 4);
  typed(t, name, at, dtype);
  const auto s = t.strides();
  if (t.size(2) != heads || t.size(3) != dim || (s[3] != 1 && dim > 1))
    value_error(std::string(name) + " must be [pages, rows, " + std::to_string(heads) + ", " + std::to_string(dim) +
                "] with contiguous columns");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) value_error(std::string(name) + " has too many pages");
  if (!values) {
    pool->num_pages = (int32_t)t.size(0);
    pool->page_size = (int32_t)t.size(1);
  } else if (t.size(0) != pool->num_pages || t.size(1) != pool->page_size) {
    value_error("k_pool and v_pool must have the same pages");
  }
  (values ? pool->v : pool->k) = t.data_ptr();
  // the stride of a dimension of one is never used and may be anything
  (values ? pool->v_page_stride : pool->k_page_stride) = t.size(0) > 1 ? s[0] : 0;
  (values ? pool->v_row_stride : pool->k_row_stride) = t.size(1) > 1 ? s[1] : 0;
  (values ? pool->v_head_stride : pool->k_head_stride) = heads > 1 ? s[2] : 0;
}

// A workspace: the caller's, or `bytes` for this call alone (its memory goes back to the stream it was used on).
void* workspace(PyObject* o, const Place& at, size_t bytes, at::Tensor* made, size_t* size) {
  if (none(o)) {
    *made = at.empty({(int64_t)std::max<size_t>(bytes, 16)}, at::kByte);
    *size = (size_t)made->numel();
    return made->data_ptr();
  }
  const at::Tensor& t = tensor(o, "workspace");
  if (t.device() != at.device || !t.is_contiguous())
    value_error("workspace must be a contiguous tensor on the first tensor's device");
  *size = t.nbytes();
  return t.data_ptr();
}

int32_t dim32(int64_t n) {
  if (n > INT32_MAX) value_error("a dimension does not fit 32 bits");
  return (int32_t)n;
}

template <typename F, typename A>
void call(F f, const A& args, const Place& at, const char* what) {
  const loza_stream_t st = at.stream();
  loza_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(&args, st);
  Py_END_ALLOW_THREADS
  if (rc != LOZA_OK) throw Status{rc, what};
}

// Runs a binding's body and turns what it throws into the Python error.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const Status& e) {
    PyObject* v = Py_BuildValue("(is)", e.code, e.what);
    if (v) {
      PyErr_SetObject(g_status_error, v);
      Py_DECREF(v);
    }
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {  // as from torch.empty: callers free memory and go on
    PyErr_SetString(g_memory_error, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) type_error("wrong number of arguments");
}

PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  bool whole = t != nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    whole = whole && o;
    if (t) PyTuple_SET_ITEM(t, i++, o); else Py_XDECREF(o);
  }
  if (whole) return t;
  Py_XDECREF(t);
  throw PythonError{};  // out of memory: already set
}

// (ctx_lens, new_lens, free_pages, block_table, page_size, capacity)
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 6);
    const at::Tensor& ctx = rank(a[0], "ctx_lens", 1);
    const Place at(ctx, "ctx_lens");
    const int64_t B = ctx.size(0);
    const at::Tensor& free = rank(a[2], "free_pages", 1);
    loza_page_plan_args p{};
    p.ctx_lens = static_cast<int32_t*>(plain(a[0], "ctx_lens", at, at::kInt, {B}));
    p.new_lens = static_cast<int32_t*>(plain(a[1], "new_lens", at, at::kInt, {B}));
    p.free_pages = static_cast<int32_t*>(plain(a[2], "free_pages", at, at::kInt, {free.size(0)}));
    const Table table(a[3], at, B);
    p.block_table = table.p;
    p.bt_stride = table.stride;
    p.batch = dim32(B);
    p.n_free = dim32(free.size(0));
    p.max_pages = dim32(table.cols);
    p.page_size = int32(a[4], "page_size");
    p.capacity = integer(a[5]);
    if (p.capacity < 0 || p.capacity > INT32_MAX) throw Status{LOZA_ERR_INVALID_ARG, "loza_page_plan"};
    at::Tensor cu = at.empty({B + 1}, at::kInt), lens = at.empty({B}, at::kInt), counts = at.empty({3}, at::kInt);
    at::Tensor pos = at.empty({p.capacity}, at::kInt), slots = at.empty({p.capacity}, at::kLong);
    p.cu_seqlens = cu.data_ptr<int32_t>();
    p.seqlens = lens.data_ptr<int32_t>();
    p.counts = counts.data_ptr<int32_t>();
    p.positions = pos.data_ptr<int32_t>();
    p.slots = slots.data_ptr<int64_t>();
    call(f_page_plan, p, at, "loza_page_plan");
    written(THPVariable_Unpack(a[3]));
    return tuple({THPVariable_Wrap(std::move(cu)), THPVariable_Wrap(std::move(lens)),
                  THPVariable_Wrap(std::move(pos)), THPVariable_Wrap(std::move(slots)),
                  THPVariable_Wrap(std::move(counts))});
  });
}

template <typename P>
void rope_tables(P* p, PyObject* positions, PyObject* inv_freq, const Place& at, int64_t tokens) {
  p->positions = static_cast<int32_t*>(plain(positions, "positions", at, at::kInt, {tokens}));
  p->inv_freq = static_cast<double*>(plain(inv_freq, "inv_freq", at, at::kDouble, {std::max(0, p->rope.rope_dim / 2)}));
}

// (x, positions, inv_freq, rope, out, transposed)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 6);
    loza_rope_args p{};
    p.rope = rope_params(a[3]);
    const at::Tensor& x = rank(a[0], "x", 3);
    const Place at(x, "x");
    p.dtype = dtype_code(x, "x");
    const int64_t T = x.size(0);
    rope_tables(&p, a[1], a[2], at, T);
    const Rows xr(x, "x", at, x.scalar_type(), x.sizes());
    Output out;
    const Rows orow = rows_out(&out, a[4], "out", at, x.scalar_type(), x.sizes());
    p.x = xr.p;
    p.x_row_stride = xr.stride;
    p.out = orow.p;
    p.out_row_stride = orow.stride;
    p.tokens = T;
    p.n_heads = dim32(x.size(1));
    p.d = dim32(x.size(2));
    const int t = PyObject_IsTrue(a[5]);
    if (t < 0) throw PythonError{};
    p.transposed = t;
    call(f_rope, p, at, "loza_rope");
    return out.take();
  });
}

// A side's weight: its address, and norm_dim (its length unless it was given).
const void* weight(PyObject* o, bool rows, const char* name, int64_t* norm_dim, const Place& at,
                   at::ScalarType dtype) {
  if (none(o)) return nullptr;
  if (!rows) value_error(std::string(name) + " without its rows");
  if (*norm_dim < 0) *norm_dim = tensor(o, name).numel();
  return plain(o, name, at, dtype, {*norm_dim});
}
int64_t given_norm_dim(PyObject* o) {
  if (none(o)) return -1;
  const int64_t v = integer(o);
  if (v < 0) value_error("norm_dim must not be negative");
  return v;
}

// (q, k, positions, inv_freq, rope, q_weight, k_weight, eps, v, k_pool, v_pool, slots, q_out, k_out, norm_dim)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 15);
    loza_qk_norm_rope_args p{};
    p.rope = rope_params(a[4]);
    const bool has_q = !none(a[0]), has_k = !none(a[1]), has_v = !none(a[8]), has_pool = !none(a[9]);
    const at::Tensor& first = has_q ? rank(a[0], "q", 3) : rank(a[1], "k", 3);
    const Place at(first, has_q ? "q" : "k");
    const at::ScalarType dtype = first.scalar_type();
    p.dtype = dtype_code(first, has_q ? "q" : "k");
    const int64_t T = first.size(0), d = first.size(2);
    p.tokens = T;
    p.d = dim32(d);
    Output q_out, k_out;
    if (has_q) {
      const Rows r(first, "q", at, dtype, first.sizes());
      const Rows o = rows_out(&q_out, a[12], "q_out", at, dtype, first.sizes());
      p.q = r.p;
      p.q_row_stride = r.stride;
      p.q_out = o.p;
      p.q_out_row_stride = o.stride;
      p.n_heads = dim32(first.size(1));
    } else if (!none(a[12])) {
      value_error("q_out without q");
    }
    if (has_k) {
      const at::Tensor& k = rank(a[1], "k", 3);
      if (k.size(0) != T || k.size(2) != d) value_error("q and k must agree in tokens and head dim");
      const Rows r(k, "k", at, dtype, k.sizes());
      p.k = r.p;
      p.k_row_stride = r.stride;
      p.n_kv_heads = dim32(k.size(1));
      if (!none(a[13]) || !has_pool) {
        const Rows o = rows_out(&k_out, a[13], "k_out", at, dtype, k.sizes());
        p.k_out = o.p;
        p.k_out_row_stride = o.stride;
      }
    } else if (!none(a[13]) || has_pool) {
      value_error("k_out and k_pool need k");
    }
    if (has_pool) {
      if (has_v == none(a[10])) value_error("v and v_pool come together");
      pool_side(&p.pool, false, a[9], at, dtype, p.n_kv_heads, d);
      p.slots = static_cast<int64_t*>(plain(a[11], "slots", at, at::kLong, {T}));
      if (has_v) {
        const at::Tensor& v = rank(a[8], "v", 3);
        if (v.size(0) != T || v.size(1) != p.n_kv_heads) value_error("v and k must agree in tokens and heads");
        const Rows r(v, "v", at, dtype, v.sizes());
        p.v = r.p;
        p.v_row_stride = r.stride;
        p.d_v = dim32(v.size(2));
        pool_side(&p.pool, true, a[10], at, dtype, p.n_kv_heads, v.size(2));
      }
    } else if (has_v || !none(a[10]) || !none(a[11])) {
      value_error("v, v_pool and slots need k_pool");
    }
    rope_tables(&p, a[2], a[3], at, T);
    int64_t norm_dim = given_norm_dim(a[14]);
    p.q_weight = weight(a[5], has_q, "q_weight", &norm_dim, at, dtype);
    p.k_weight = weight(a[6], has_k, "k_weight", &norm_dim, at, dtype);
    p.norm_dim = dim32(std::max<int64_t>(0, norm_dim));
    p.eps = (float)number(a[7]);
    call(f_norm_rope, p, at, "loza_qk_norm_rope");
    if (has_pool) written(THPVariable_Unpack(a[9]));
    if (has_pool && has_v) written(THPVariable_Unpack(a[10]));
    return tuple({q_out.take(), k_out.take()});
  });
}

// (dq_out, dk_out, q, k, positions, inv_freq, rope, q_weight, k_weight, eps, dq, dk, norm_dim, workspace)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 14);
    loza_qk_norm_rope_backward_args p{};
    p.rope = rope_params(a[6]);
    const bool has_q = !none(a[0]), has_k = !none(a[1]);
    const at::Tensor& first = has_q ? rank(a[0], "dq_out", 3) : rank(a[1], "dk_out", 3);
    const Place at(first, has_q ? "dq_out" : "dk_out");
    const at::ScalarType dtype = first.scalar_type();
    p.dtype = dtype_code(first, has_q ? "dq_out" : "dk_out");
    const int64_t T = first.size(0), d = first.size(2);
    p.tokens = T;
    p.d = dim32(d);
    int64_t norm_dim = given_norm_dim(a[12]);
    p.q_weight = weight(a[7], has_q, "q_weight", &norm_dim, at, dtype);
    p.k_weight = weight(a[8], has_k, "k_weight", &norm_dim, at, dtype);
    p.norm_dim = dim32(std::max<int64_t>(0, norm_dim));
    Output dq, dk;
    at::Tensor dqw, dkw, ws;
    if (has_q) {
      const Rows g(first, "dq_out", at, dtype, first.sizes());
      const Rows o = rows_out(&dq, a[10], "dq", at, dtype, first.sizes());
      p.dq_out = g.p;
      p.dq_out_row_stride = g.stride;
      p.dq = o.p;
      p.dq_row_stride = o.stride;
      p.n_heads = dim32(first.size(1));
      if (p.q_weight) {
        const Rows r(tensor(a[2], "q"), "q", at, dtype, first.sizes());
        p.q = r.p;
        p.q_row_stride = r.stride;
        dqw = at.empty({norm_dim}, at::kFloat);
        p.dq_weight = dqw.data_ptr<float>();
      }
    } else if (!none(a[10])) {
      value_error("dq without dq_out");
    }
    if (has_k) {
      const at::Tensor& gk = rank(a[1], "dk_out", 3);
      if (gk.size(0) != T || gk.size(2) != d) value_error("dq_out and dk_out must agree in tokens and head dim");
      const Rows g(gk, "dk_out", at, dtype, gk.sizes());
      const Rows o = rows_out(&dk, a[11], "dk", at, dtype, gk.sizes());
      p.dk_out = g.p;
      p.dk_out_row_stride = g.stride;
      p.dk = o.p;
      p.dk_row_stride = o.stride;
      p.n_kv_heads = dim32(gk.size(1));
      if (p.k_weight) {
        const Rows r(tensor(a[3], "k"), "k", at, dtype, gk.sizes());
        p.k = r.p;
        p.k_row_stride = r.stride;
        dkw = at.empty({norm_dim}, at::kFloat);
        p.dk_weight = dkw.data_ptr<float>();
      }
    } else if (!none(a[11])) {
      value_error("dk without dk_out");
    }
    rope_tables(&p, a[4], a[5], at, T);
    p.eps = (float)number(a[9]);
    if (p.q_weight || p.k_weight)
      p.workspace = workspace(a[13], at, f_norm_rope_workspace(p.norm_dim), &ws, &p.workspace_bytes);
    call(f_norm_rope_backward, p, at, "loza_qk_norm_rope_backward");
    auto wrap = [](at::Tensor& t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None); };
    return tuple({dq.take(), dk.take(), wrap(dqw), wrap(dkw)});
  });
}

// (q, k_pool, v_pool, block_table, seqlens, max_seqlen, params, out, lse, workspace)
PyObject* decode_paged_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 10);
    loza_decode_paged_kv_args p{};
    p.window = params<loza_ssa_params>(a[6], g_window_params, "params must be a Params");
    const at::Tensor& q = rank(a[0], "q", 3);
    const Place at(q, "q");
    const at::ScalarType dtype = q.scalar_type();
    p.dtype = dtype_code(q, "q");
    const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
    const Rows r(q, "q", at, dtype, q.sizes());
    p.q = r.p;
    p.q_row_stride = r.stride;
    p.batch = dim32(B);
    p.n_heads = dim32(H);
    p.d_qk = dim32(d);
    p.n_kv_heads = dim32(rank(a[1], "k_pool", 4).size(2));
    p.d_v = dim32(rank(a[2], "v_pool", 4).size(3));
    pool_side(&p.pool, false, a[1], at, dtype, p.n_kv_heads, d);
    pool_side(&p.pool, true, a[2], at, dtype, p.n_kv_heads, p.d_v);
    const Table table(a[3], at, B);
    p.block_table = table.p;
    p.bt_stride = table.stride;
    p.seqlens = static_cast<int32_t*>(plain(a[4], "seqlens", at, at::kInt, {B}));
    p.max_seqlen = int32(a[5], "max_seqlen");
    if (table.cols * p.pool.page_size < p.max_seqlen) value_error("block_table has too few columns for max_seqlen");
    Output out, lse;
    at::Tensor ws;
    if (none(a[7])) {
      out.made = at.empty({B, H, p.d_v}, dtype);
      p.out = out.made.data_ptr();
    } else {
      out.given = a[7];
      p.out = plain(a[7], "out", at, dtype, {B, H, p.d_v});
    }
    if (none(a[8])) {
      lse.made = at.empty({B, H}, at::kFloat);
      p.lse = lse.made.data_ptr<float>();
    } else {
      lse.given = a[8];
      p.lse = static_cast<float*>(plain(a[8], "lse", at, at::kFloat, {B, H}));
    }
    p.workspace = workspace(a[9], at, f_decode_workspace(p.n_heads, p.n_kv_heads, p.d_qk, p.d_v), &ws,
                            &p.workspace_bytes);
    call(f_decode, p, at, "loza_ssa_decode_paged_kv");
    return tuple({out.take(), lse.take()});
  });
}

// ({name: address}, LozaError, RopeParams, Params, torch.OutOfMemoryError)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 5);
    auto at = [&](const char* name) {
      PyObject* v = PyDict_Check(a[0]) ? PyDict_GetItemString(a[0], name) : nullptr;
      if (!v) type_error(std::string("no address of ") + name);
      return reinterpret_cast<void*>(integer(v));
    };
    f_page_plan = reinterpret_cast<decltype(f_page_plan)>(at("loza_page_plan"));
    f_rope = reinterpret_cast<decltype(f_rope)>(at("loza_rope"));
    f_norm_rope = reinterpret_cast<decltype(f_norm_rope)>(at("loza_qk_norm_rope"));
    f_norm_rope_backward = reinterpret_cast<decltype(f_norm_rope_backward)>(at("loza_qk_norm_rope_backward"));
    f_norm_rope_workspace = reinterpret_cast<decltype(f_norm_rope_workspace)>(at("loza_qk_norm_rope_workspace_size"));
    f_decode = reinterpret_cast<decltype(f_decode)>(at("loza_ssa_decode_paged_kv"));
    f_decode_workspace = reinterpret_cast<decltype(f_decode_workspace)>(at("loza_decode_paged_kv_workspace_size"));
    g_status_error = Py_NewRef(a[1]);
    g_rope_params = Py_NewRef(a[2]);
    g_window_params = Py_NewRef(a[3]);
    g_memory_error = Py_NewRef(a[4]);
    return Py_NewRef(Py_None);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind>("bind"), method<page_plan>("page_plan"), method<rope>("rope"),
                           method<qk_norm_rope>("qk_norm_rope"),
                           method<qk_norm_rope_backward>("qk_norm_rope_backward"),
                           method<decode_paged_kv>("decode_paged_kv"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", LOZA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
