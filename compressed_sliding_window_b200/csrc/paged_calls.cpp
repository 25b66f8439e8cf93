// Fast path of the Python binding of the paged cache (include/hca.h, "Paged
// cache" and "Pages"): checks the tensors of a call and makes it, without the
// interpreter touching them one by one (a serving step has a dozen: 12 of its
// 20 us on the host).  A call whose arguments are not exactly what the library
// takes is not made: the function returns False, and the Python code above
// finds out what is wrong and says it.  No computation here.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/torch.h>

#include <cmath>
#include <initializer_list>

#include "../../include/hca.h"

namespace {

constexpr int64_t kDim = HCA_HEAD_DIM, kHeads = HCA_NUM_HEADS, kWin = HCA_WINDOW;

// The tensor behind a Python object, or null.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Checks the tensors of one call; `good` ends false when one is not as needed.
struct Args {
  c10::Device device{c10::DeviceType::CPU};
  bool good = true;

  void* need(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(o);
    if (t == nullptr || t->scalar_type() != type || t->device() != device ||
        t->sizes() != at::IntArrayRef(shape.begin(), shape.size()) || !t->is_contiguous() ||
        t->layout() != at::kStrided) {
      good = false;
      return nullptr;
    }
    return t->numel() > 0 ? t->data_ptr() : nullptr;
  }
  hca_bf16* bf16(PyObject* o, std::initializer_list<int64_t> shape) {
    return static_cast<hca_bf16*>(need(o, at::kBFloat16, shape));
  }
  int32_t* ints(PyObject* o, std::initializer_list<int64_t> shape) {
    return static_cast<int32_t*>(need(o, at::kInt, shape));
  }
  // sets the device of the call
  bool on(PyObject* o) {
    const at::Tensor* t = tensor(o);
    good = t != nullptr && t->is_cuda();
    if (good) device = t->device();
    return good;
  }
  int64_t size(PyObject* o, int dim, int64_t dims) {
    const at::Tensor* t = tensor(o);
    if (t == nullptr || t->dim() != dims) {
      good = false;
      return 0;
    }
    return t->size(dim);
  }
  // [rows, max_pages] int32, rows possibly apart
  int32_t* table(PyObject* o, int64_t rows, int64_t& cols, int64_t& stride) {
    const at::Tensor* t = tensor(o);
    if (t == nullptr || t->scalar_type() != at::kInt || t->device() != device || t->dim() != 2 ||
        t->size(0) != rows) {
      good = false;
      return nullptr;
    }
    cols = t->size(1);
    stride = rows > 1 ? t->stride(0) : cols;
    if ((cols > 1 && t->stride(1) != 1) || stride < cols) good = false;
    return cols > 0 && rows > 0 ? t->data_ptr<int32_t>() : nullptr;
  }
  void cache(hca_paged_cache_t& c, int64_t S, PyObject* wk, PyObject* wv, PyObject* ws,
             PyObject* ck, PyObject* cv, PyObject* page_table) {
    c.wk = bf16(wk, {S, kWin, kDim});
    c.wv = bf16(wv, {S, kWin, kDim});
    c.ws = ws == Py_None ? nullptr : bf16(ws, {S, kWin});
    const int64_t num = size(ck, 0, 3), page = size(ck, 1, 3);
    c.ck = bf16(ck, {num, page, kDim});
    c.cv = bf16(cv, {num, page, kDim});
    int64_t cols = 0, stride = 0;
    c.page_table = table(page_table, S, cols, stride);
    c.table_stride = stride;
    good = good && num <= INT_MAX && cols <= INT_MAX;
    c.max_pages = static_cast<int>(cols);
    c.num_pages = static_cast<int>(num);
    c.page_size = static_cast<int>(page);
  }
  void pages(hca_page_table_t& p, PyObject* page_table, PyObject* n_pages, PyObject* ref,
             PyObject* page_size) {
    const int64_t rows = size(n_pages, 0, 1), num = size(ref, 0, 1);
    p.n_pages = ints(n_pages, {rows});
    p.ref = ints(ref, {num});
    int64_t cols = 0, stride = 0;
    p.page_table = table(page_table, rows, cols, stride);
    p.table_stride = stride;
    good = good && num <= INT_MAX && cols <= INT_MAX && rows <= INT_MAX && PyLong_Check(page_size);
    p.rows = static_cast<int>(rows);
    p.max_pages = static_cast<int>(cols);
    p.num_pages = static_cast<int>(num);
    int overflow = 0;
    const long size = good ? PyLong_AsLongAndOverflow(page_size, &overflow) : 0;
    good = good && overflow == 0 && size >= 0 && size <= INT_MAX;
    p.page_size = static_cast<int>(size);
  }
  // a tuple or list of [items, ...] tensors appended to out[n ..]
  int arrays(PyObject* seq, int64_t items, hca_page_array_t* out, int n, int most) {
    if (!PyTuple_Check(seq) && !PyList_Check(seq)) {
      good = false;
      return n;
    }
    const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
    for (Py_ssize_t i = 0; i < len && good; ++i) {
      const at::Tensor* t = tensor(PySequence_Fast_GET_ITEM(seq, i));
      if (n >= most || t == nullptr || t->device() != device || !t->is_contiguous() ||
          t->dim() < 2 || t->size(0) != items || items < 1) {
        good = false;
        return n;
      }
      const int64_t bytes = static_cast<int64_t>(t->nbytes()) / items;
      if (bytes < 16 || bytes % 16 != 0) {
        good = false;
        return n;
      }
      out[n++] = {t->data_ptr(), bytes};
    }
    return n;
  }
};

// workspace given, or none
void* bytes_of(Args& a, PyObject* o, size_t& size) {
  const int64_t n = a.size(o, 0, 1);
  size = static_cast<size_t>(n);
  return a.need(o, at::kByte, {n});
}

cudaStream_t stream_of(const Args& a) {
  return c10::cuda::getCurrentCUDAStream(a.device.index()).stream();
}

at::Tensor fresh(const Args& a, at::ScalarType type, int64_t n) {
  return at::empty({n}, at::TensorOptions().dtype(type).device(a.device));
}

// What a call returns: False (arguments to be looked at), a status code, or `value`.
PyObject* refused() { Py_RETURN_FALSE; }
PyObject* answer(hca_status_t st, PyObject* value) {
  if (st == HCA_OK) return value;
  Py_XDECREF(value);
  return PyLong_FromLong(st);
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

using Fast = PyObject* (*)(PyObject* const*, Py_ssize_t);
// No C++ exception leaves a call: torch's own become the Python ones that the same
// allocation would raise there (torch.OutOfMemoryError for one).
template <Fast kCall, Py_ssize_t kArgs>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  HANDLE_TH_ERRORS
  return kCall(args, n);
  END_HANDLE_TH_ERRORS
}

// k_new, v_new, s_new, q_start | None, ctx_len, wk, wv, ws, ck, cv, table
PyObject* paged_append(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[5])) return refused();
  const int64_t S = a.size(v[4], 0, 1), N = a.size(v[0], 0, 2);
  const auto* len = a.ints(v[4], {S});
  const auto* k = a.bf16(v[0], {N, kDim});
  const auto* vv = a.bf16(v[1], {N, kDim});
  const auto* s = a.bf16(v[2], {N});
  const auto* start = v[3] == Py_None ? nullptr : a.ints(v[3], {S + 1});
  hca_paged_cache_t c;
  a.cache(c, S, v[5], v[6], v[7], v[8], v[9], v[10]);
  if (!a.good || N < 1 || N > INT_MAX || S > INT_MAX) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  return answer(hca_paged_append(k, vv, s, start, len, static_cast<int>(S), static_cast<int>(N), &c,
                                 stream_of(a)),
                none());
}

// The attention's own arguments: q, g, out | None, workspace, scale | None.
struct Attend {
  const hca_bf16 *q, *g;
  hca_bf16* out;
  PyObject* out_object = nullptr;
  void* ws;
  size_t ws_bytes;
  float scale;

  bool take(Args& a, int64_t rows, PyObject* q_, PyObject* g_, PyObject* out_, PyObject* ws_,
            PyObject* scale_) {
    q = a.bf16(q_, {rows, kHeads, kDim});
    g = a.bf16(g_, {rows, kHeads, kDim});
    ws = bytes_of(a, ws_, ws_bytes);
    scale = 1.0f / std::sqrt(static_cast<float>(kDim));
    if (scale_ != Py_None) {
      if (!PyFloat_Check(scale_)) return false;
      scale = static_cast<float>(PyFloat_AS_DOUBLE(scale_));
    }
    if (out_ != Py_None) {
      out = a.bf16(out_, {rows, kHeads, kDim});
      if (!a.good) return false;
      Py_INCREF(out_);
      out_object = out_;
    } else {
      if (!a.good) return false;
      at::Tensor t = at::empty({rows, kHeads, kDim},
                               at::TensorOptions().dtype(at::kBFloat16).device(a.device));
      out = static_cast<hca_bf16*>(t.data_ptr());
      out_object = THPVariable_Wrap(std::move(t));
    }
    return out_object != nullptr;
  }
};

// q, g, k_new, v_new, s_new, q_start, ctx_len, wk, wv, ws, ck, cv, table, scale, workspace, out
PyObject* paged_prefill(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[7])) return refused();
  const int64_t S = a.size(v[6], 0, 1), N = a.size(v[2], 0, 2);
  const auto* len = a.ints(v[6], {S});
  const auto* k = a.bf16(v[2], {N, kDim});
  const auto* vv = a.bf16(v[3], {N, kDim});
  const auto* s = a.bf16(v[4], {N});
  const auto* start = a.ints(v[5], {S + 1});
  hca_paged_cache_t c;
  a.cache(c, S, v[7], v[8], v[9], v[10], v[11], v[12]);
  if (!a.good || N < 1 || N > INT_MAX || S > INT_MAX) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  Attend t;
  if (!t.take(a, N, v[0], v[1], v[15], v[14], v[13])) return refused();
  return answer(hca_paged_prefill(t.q, t.g, k, vv, s, start, len, static_cast<int>(S),
                                  static_cast<int>(N), kHeads, t.scale, nullptr, nullptr, 0, &c,
                                  t.out, t.ws, t.ws_bytes, stream_of(a)),
                t.out_object);
}

// q, ck, cv, table, wk, wv, ctx_len, g, scale, workspace, out
PyObject* paged_decode(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[4])) return refused();
  const int64_t S = a.size(v[6], 0, 1);
  const auto* len = a.ints(v[6], {S});
  hca_paged_cache_t c;
  a.cache(c, S, v[4], v[5], Py_None, v[1], v[2], v[3]);
  if (!a.good || S > INT_MAX) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  Attend t;
  if (!t.take(a, S, v[0], v[7], v[10], v[9], v[8])) return refused();
  return answer(hca_paged_decode(t.q, t.g, len, static_cast<int>(S), kHeads, t.scale, nullptr,
                                 nullptr, 0, &c, t.out, t.ws, t.ws_bytes, stream_of(a)),
                t.out_object);
}

// q, g, k_new, v_new, s_new, ctx_len, wk, wv, ws, ck, cv, table, scale, workspace, out
PyObject* paged_decode_step(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[6])) return refused();
  const int64_t S = a.size(v[5], 0, 1);
  const auto* len = a.ints(v[5], {S});
  const auto* k = a.bf16(v[2], {S, kDim});
  const auto* vv = a.bf16(v[3], {S, kDim});
  const auto* s = a.bf16(v[4], {S});
  hca_paged_cache_t c;
  a.cache(c, S, v[6], v[7], v[8], v[9], v[10], v[11]);
  if (!a.good || S > INT_MAX) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  Attend t;
  if (!t.take(a, S, v[0], v[1], v[14], v[13], v[12])) return refused();
  return answer(hca_paged_decode_step(t.q, t.g, k, vv, s, len, static_cast<int>(S), kHeads, t.scale,
                                      nullptr, nullptr, 0, &c, t.out, t.ws, t.ws_bytes,
                                      stream_of(a)),
                t.out_object);
}

// A page operation's workspace: the caller's, or `n` fresh bytes held by `own`.
void* room(Args& a, PyObject* o, int rows, int pages, int n, at::Tensor& own, size_t& size) {
  if (o != Py_None) return bytes_of(a, o, size);
  size = hca_pages_workspace_size(rows, pages, n);
  own = fresh(a, at::kByte, static_cast<int64_t>(size));
  return own.data_ptr();
}

// table, n_pages, ref, entries, page_size, workspace | None
PyObject* resize_pages(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[0])) return refused();
  hca_page_table_t p;
  a.pages(p, v[0], v[1], v[2], v[4]);
  const auto* entries = a.ints(v[3], {p.rows});
  if (!a.good) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  at::Tensor own;
  size_t size;
  void* ws = room(a, v[5], p.rows, p.num_pages, 0, own, size);
  if (!a.good) return refused();
  return answer(hca_pages_resize(&p, entries, ws, size, stream_of(a)), none());
}

// table, n_pages, ref, parents, children, entries, pools, page_size, rings, workspace | None
PyObject* fork_pages(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[0])) return refused();
  hca_page_table_t p;
  a.pages(p, v[0], v[1], v[2], v[7]);
  const int64_t n = a.size(v[3], 0, 1);
  const auto* parents = a.ints(v[3], {n});
  const auto* children = a.ints(v[4], {n});
  const auto* entries = a.ints(v[5], {n});
  hca_page_array_t arrays[8];
  const int pools = a.arrays(v[6], p.num_pages, arrays, 0, 8);
  const int all = a.arrays(v[8], p.rows, arrays, pools, 8);
  if (!a.good || n < 1 || n > INT_MAX) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  at::Tensor own, ok = fresh(a, at::kInt, n);
  size_t size;
  void* ws = room(a, v[9], p.rows, p.num_pages, static_cast<int>(n), own, size);
  if (!a.good) return refused();
  const hca_status_t st =
      hca_pages_fork(&p, parents, children, entries, static_cast<int>(n), arrays, pools,
                     arrays + pools, all - pools, ok.data_ptr<int32_t>(), ws, size, stream_of(a));
  return answer(st, THPVariable_Wrap(std::move(ok)));
}

// table, n_pages, ref, pools, page_size, workspace | None
PyObject* compact_pages(PyObject* const* v, Py_ssize_t) {
  Args a;
  if (!a.on(v[0])) return refused();
  hca_page_table_t p;
  a.pages(p, v[0], v[1], v[2], v[4]);
  hca_page_array_t arrays[8];
  const int pools = a.arrays(v[3], p.num_pages, arrays, 0, 8);
  if (!a.good) return refused();
  const c10::cuda::OptionalCUDAGuard guard(a.device);
  at::Tensor own, live = fresh(a, at::kInt, 1);
  size_t size;
  void* ws = room(a, v[5], p.rows, p.num_pages, 0, own, size);
  if (!a.good) return refused();
  const hca_status_t st = hca_pages_compact(&p, arrays, pools, live.data_ptr<int32_t>(), ws, size,
                                            stream_of(a));
  return answer(st, THPVariable_Wrap(std::move(live)));
}

#define CALL(name, args)                                                                     \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name, args>)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(paged_append, 11),      CALL(paged_prefill, 16),
                         CALL(paged_decode, 11),      CALL(paged_decode_step, 15),
                         CALL(resize_pages, 6),       CALL(fork_pages, 10),
                         CALL(compact_pages, 6),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_calls(void) {
  PyObject* m = PyModule_Create(&module);
  // the torch that it was built against; the binding compares
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", HCA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
