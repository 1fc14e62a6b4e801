// The paged cache's calls from Python: checks of the tensors and marshalling of
// their pointers, shapes and strides into the C ABI.  These calls run once per
// layer and token; through ctypes their 10 to 35 arguments cost more host time
// than the launch (append of one token 12 us a call, 5 of them in the library).
//
// A refused tensor raises AssertionError, one on another device than the
// current one ValueError, an error status of the library its MLAError; nothing
// has then been launched.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "mla.h"

namespace {

PyObject* g_error = nullptr;        // MLAError(status, detail)
PyObject* g_get_device = nullptr;   // the current CUDA device
PyObject* g_raw_stream = nullptr;   // its current stream's handle

struct Refused {
  PyObject* type;       // null: a Python error is set already
  const char* message;
};
#define NEED(cond, message) \
  do {                      \
    if (!(cond)) throw Refused{PyExc_AssertionError, message}; \
  } while (0)

using Tensor = at::Tensor;

const Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, "a torch tensor is expected"};
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

template <typename T>
T* data(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T>
T* data(const Tensor* t) { return t ? data<T>(*t) : nullptr; }

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, nullptr};
  return v;
}
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) throw Refused{PyExc_OverflowError, "a size that does not fit 32 bits"};
  return (int32_t)v;
}
int32_t size32(int64_t v) {
  NEED(v == (int32_t)v, "a size that does not fit 32 bits");
  return (int32_t)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, nullptr};
  return (float)v;
}

int dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return MLA_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return MLA_DTYPE_BF16;
  throw Refused{PyExc_TypeError, "unsupported dtype (float32 and bfloat16 are served)"};
}

// Lengths, counts and positions that the kernels read or write `count` of.
void need_int32(const Tensor* t, int64_t count) {
  NEED(!t || (t->scalar_type() == at::kInt && t->is_contiguous() && t->numel() >= count),
       "lengths, counts and positions: contiguous int32, at least one for each row");
}
void need_status(const Tensor* t) {
  NEED(!t || t->numel() * (int64_t)t->element_size() >= 4, "device_status: one int32");
}

struct Pool {
  int32_t pages, page_size, features;
  int64_t row, page;
  explicit Pool(const Tensor& t) {
    NEED(t.dim() == 3 && t.stride(2) == 1, "pools: [num_pages, page_size, features], the last axis contiguous");
    pages = size32(t.size(0)), page_size = size32(t.size(1)), features = size32(t.size(2));
    page = t.stride(0), row = t.stride(1);
  }
};
struct Table {
  int32_t* data;
  int64_t row;
  int32_t width;
  Table(const Tensor& t, int64_t batch) {
    NEED(t.dim() == 2 && t.scalar_type() == at::kInt && t.stride(1) == 1 && t.size(0) >= batch,
         "page_table: [>= batch, width] int32, rows contiguous");
    data = ::data<int32_t>(t), row = t.stride(0), width = size32(t.size(1));
  }
};

// The launch stream's handle, once every tensor is known to live on the current device.
template <typename... Ts>
mla_stream_t stream_for(PyObject* stream, const int64_t* device_of_arrays, Ts... tensors) {
  PyObject* d = PyObject_CallNoArgs(g_get_device);
  if (!d) throw Refused{nullptr, nullptr};
  const long device = PyLong_AsLong(d);
  bool same = !device_of_arrays || *device_of_arrays == device;
  ((same = same && (!tensors || tensors->get_device() == device)), ...);
  PyObject* handle = !same ? nullptr : stream == Py_None ? PyObject_CallOneArg(g_raw_stream, d)
                                                         : PyObject_GetAttrString(stream, "cuda_stream");
  Py_DECREF(d);
  if (!same) throw Refused{PyExc_ValueError, "a tensor that is not on the current CUDA device"};
  if (!handle) throw Refused{nullptr, nullptr};
  void* p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (!p && PyErr_Occurred()) throw Refused{nullptr, nullptr};
  return static_cast<mla_stream_t>(p);
}

// The interpreter's lock is released during a call of the library: its launches wait while the stream's queue is full,
// and what empties that queue may need another Python thread.
template <typename F>
int unlocked(F&& call) {
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return call();
}

PyObject* finish(int status) {
  if (status == MLA_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, mla_last_error_detail());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// No C++ exception leaves a Python entry.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t expected, F&& f) {
  if (n != expected) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", expected, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.message);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Tensor &raw = tensor(a[0]), &raw_rope = tensor(a[1]), &gain = tensor(a[2]);
    const float eps = real(a[3]), theta = real(a[4]);
    const Tensor &latent = tensor(a[5]), &rope = tensor(a[6]), &table = tensor(a[7]), &len = tensor(a[8]);
    const Tensor *out = optional(a[9]), *positions = optional(a[10]), *counts = optional(a[11]), *status = optional(a[12]);
    NEED(raw.dim() == 3 && raw_rope.dim() == 3 && raw.stride(2) == 1 && raw_rope.stride(2) == 1,
         "new tokens: [batch, tokens, features], the last axis contiguous");
    const int64_t batch = raw.size(0), s = raw.size(1), rank = raw.size(2);
    const Pool l(latent), r(rope);
    const Table t(table, batch);
    NEED(gain.is_contiguous() && gain.numel() == rank && l.features == rank, "norm_weight and the pool: one rank");
    NEED(raw_rope.scalar_type() == raw.scalar_type() && gain.scalar_type() == raw.scalar_type() &&
             raw_rope.size(0) == batch && raw_rope.size(1) == s && raw_rope.size(2) == r.features,
         "rope_raw and norm_weight: the type of latent_raw, and its tokens");
    NEED(r.pages == l.pages && r.page_size == l.page_size && rope.scalar_type() == latent.scalar_type(),
         "latent and rope pools: the same pages and type");
    need_int32(&len, batch);
    need_int32(out, batch);
    need_int32(counts, batch);
    need_int32(positions, batch * s);
    need_status(status);
    const mla_stream_t stream = stream_for(a[13], nullptr, &raw, &raw_rope, &gain, &latent, &rope, &table, &len, out, positions, counts, status);
    return finish(unlocked([&] {
      return mla_append_paged(
          raw.data_ptr(), raw.stride(0), raw.stride(1), raw_rope.data_ptr(), raw_rope.stride(0), raw_rope.stride(1),
          dtype_of(raw), gain.data_ptr(), eps, theta, data<int32_t>(positions), latent.data_ptr(), l.row, l.page,
          rope.data_ptr(), r.row, r.page, dtype_of(latent), t.data, t.row, t.width, l.page_size, l.pages,
          data<int32_t>(len), data<int32_t>(counts), data<int32_t>(out), size32(batch), size32(s), size32(rank), r.features,
          data<int32_t>(status), stream);
    }));
  });
}

PyObject* tree_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Tensor& parents = tensor(a[0]);
    const Tensor* len = optional(a[1]);
    const Tensor &positions = tensor(a[2]), &mask = tensor(a[3]);
    const Tensor *counts = optional(a[4]), *status = optional(a[5]);
    NEED(parents.dim() == 2 && parents.scalar_type() == at::kInt && parents.stride(1) == 1,
         "parents: [batch, nodes] int32, rows contiguous");
    const int64_t batch = parents.size(0), nodes = parents.size(1);
    NEED(mask.scalar_type() == at::kLong && mask.is_contiguous() && mask.numel() >= batch * nodes * ((nodes + 63) / 64),
         "tree_mask: contiguous int64, ceil(nodes / 64) words for each node");
    need_int32(len, batch);
    need_int32(counts, batch);
    need_int32(&positions, batch * nodes);
    need_status(status);
    const mla_stream_t stream = stream_for(a[6], nullptr, &parents, len, &positions, &mask, counts, status);
    return finish(unlocked([&] {
      return mla_tree_plan(data<int32_t>(parents), parents.stride(0), data<int32_t>(len), data<int32_t>(counts),
                           size32(batch), size32(nodes), data<int32_t>(positions), data<uint64_t>(mask),
                           data<int32_t>(status), stream);
    }));
  });
}

PyObject* decode_attend_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    const Tensor &q = tensor(a[0]), &latent = tensor(a[1]), &rope = tensor(a[2]), &table = tensor(a[3]), &len = tensor(a[4]);
    const int32_t batch = integer32(a[5]), s = integer32(a[6]);
    const float scale = real(a[7]);
    const Tensor& ctx = tensor(a[8]);
    const Tensor *lse = optional(a[9]), *counts = optional(a[10]), *mask = optional(a[11]), *sel = optional(a[12]),
                 *sel_count = optional(a[13]);
    const Tensor& ws = tensor(a[14]);
    const Tensor* status = optional(a[15]);
    const Pool l(latent), r(rope);
    const Table t(table, batch);
    const int64_t n_q = (int64_t)batch * s;
    NEED(q.dim() == 3 && ctx.dim() == 3 && q.stride(2) == 1 && ctx.stride(2) == 1 && q.size(0) == n_q &&
             q.size(2) == (int64_t)l.features + r.features,
         "q: [batch * s_q, heads, rank + rope_dim], the last axis contiguous");
    const int64_t heads = q.size(1);
    NEED(ctx.size(0) == n_q && ctx.size(1) == heads && ctx.size(2) == l.features, "ctx_out: [batch * s_q, heads, rank]");
    NEED(rope.scalar_type() == q.scalar_type() && latent.scalar_type() == q.scalar_type() && r.pages == l.pages &&
             r.page_size == l.page_size,
         "latent and rope pools: the query's type, the same pages");
    need_int32(&len, batch);
    need_int32(counts, batch);
    need_status(status);
    NEED(!lse || (lse->scalar_type() == at::kFloat && lse->is_contiguous() && lse->numel() == n_q * heads),
         "lse_out: contiguous float32, one for each query row and head");
    NEED(!mask || (mask->scalar_type() == at::kLong && mask->is_contiguous() && mask->numel() >= n_q * ((s + 63) / 64)),
         "tree_mask: contiguous int64, ceil(s_q / 64) words for each query row");
    int32_t k_max = 0;
    if (sel) {
      NEED(sel->dim() == 2 && sel->size(0) == n_q && sel_count && sel_count->numel() == n_q,
           "sel: [batch * s_q, k_max], with a count for each row");
      need_int32(sel, n_q);
      need_int32(sel_count, n_q);
      k_max = size32(sel->size(1));
    }
    NEED(ws.element_size() == 1 && ws.is_contiguous(), "workspace: contiguous bytes");
    const mla_stream_t stream =
        stream_for(a[16], nullptr, &q, &latent, &rope, &table, &len, &ctx, lse, counts, mask, sel, sel_count, &ws, status);
    return finish(unlocked([&] {
      return mla_decode_attend_paged(
          q.data_ptr(), q.stride(0), q.stride(1), latent.data_ptr(), l.row, l.page, rope.data_ptr(), r.row, r.page,
          dtype_of(q), t.data, t.row, t.width, l.page_size, l.pages, data<int32_t>(len), data<int32_t>(counts),
          data<uint64_t>(mask), batch, s, size32(heads), l.features, r.features, data<int32_t>(sel),
          sel ? data<int32_t>(sel_count) : nullptr, k_max, scale, ctx.data_ptr(), ctx.stride(0), ctx.stride(1), dtype_of(ctx),
          data<float>(lse), ws.data_ptr(), (size_t)ws.numel(), data<int32_t>(status), stream);
    }));
  });
}

PyObject* commit_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const auto* arrays = static_cast<const mla_state_array*>(PyLong_AsVoidPtr(a[0]));
    if (!arrays && PyErr_Occurred()) throw Refused{nullptr, nullptr};
    const int32_t n_arrays = integer32(a[1]), pages = integer32(a[2]), page_size = integer32(a[3]);
    const int64_t device = integer(a[4]);
    const Tensor &table = tensor(a[5]), &len = tensor(a[6]), &path = tensor(a[7]), &counts = tensor(a[8]);
    const Tensor *out = optional(a[9]), *status = optional(a[10]);
    NEED(path.dim() == 2 && path.scalar_type() == at::kInt && path.stride(1) == 1, "path: [batch, width] int32, rows contiguous");
    const int64_t batch = path.size(0);
    const Table t(table, batch);
    need_int32(&len, batch);
    need_int32(&counts, batch);
    need_int32(out, batch);
    need_status(status);
    const mla_stream_t stream = stream_for(a[11], &device, &table, &len, &path, &counts, out, status);
    return finish(unlocked([&] {
      return mla_commit_paged(arrays, n_arrays, t.data, t.row, t.width, page_size, pages, data<int32_t>(len),
                              data<int32_t>(path), path.stride(0), size32(path.size(1)), data<int32_t>(counts),
                              data<int32_t>(out), size32(batch), data<int32_t>(status), stream);
    }));
  });
}

PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Py_XSETREF(g_error, Py_NewRef(a[0]));
    Py_XSETREF(g_get_device, Py_NewRef(a[1]));
    Py_XSETREF(g_raw_stream, Py_NewRef(a[2]));
    Py_RETURN_NONE;
  });
}

#define FAST(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(setup), FAST(append_paged), FAST(tree_plan), FAST(decode_attend_paged), FAST(commit_paged),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
