// paged_binding.cpp — CPython entry points of the paged cache's torch helpers for
// the ordinary call: operands of the right type, layout and shape on the current
// device, work on its current stream, outputs allocated here.  A decoding step
// makes several of these calls for every layer, and checking ten operands through
// Python attributes costs more than the kernels of a short call.
//
// Each function checks its operands, allocates outputs, calls the C entry point of
// include/fa.h and returns its result (or the status, an int, where that is not
// FA_OK).  It returns None where the call is not the ordinary one; the Python
// helper then says what is wrong, or changes device, and calls the same C entry
// point itself.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>

#include "../../include/fa.h"

namespace {

decltype(&fa_cache_append) g_append;
decltype(&fa_fwd_paged_workspace_bytes) g_paged_bytes;
decltype(&fa_fwd_paged) g_paged;
decltype(&fa_cache_compact) g_compact;
decltype(&fa_cache_fork) g_fork;
decltype(&fa_cache_resize_workspace_bytes) g_resize_bytes;
decltype(&fa_cache_resize) g_resize;

// The operands of one call: each `take` returns the tensor if it is a dense CUDA
// tensor of this type and rank on the device of the first one, and clears ok if not.
struct Operands {
  bool ok = true;
  int device = -1;
  const at::Tensor *take(PyObject *x, at::ScalarType type, int64_t lo, int64_t hi) {
    if (!ok || !THPVariable_Check(x)) return fail();
    const at::Tensor &t = THPVariable_Unpack(x);
    if (!t.is_cuda() || t.scalar_type() != type || t.dim() < lo || t.dim() > hi || t.layout() != at::kStrided ||
        !t.is_contiguous())
      return fail();
    if (device < 0) device = t.get_device();
    if (t.get_device() != device) return fail();
    for (const int64_t n : t.sizes())
      if (n > INT_MAX) return fail();
    return &t;
  }
  const at::Tensor *fail() {
    ok = false;
    return nullptr;
  }
  bool current() const { return ok && device == c10::cuda::current_device(); }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

int size(const at::Tensor *t, int64_t i) { return (int)t->size(i); }
int *ints(const at::Tensor *t) { return static_cast<int *>(t->data_ptr()); }

// k_pages, v_pages, page_table, cache_lens of a call.
struct Cache {
  const at::Tensor *k, *v, *table, *lens;
  int layers = 1, num_pages, page_size, Hkv, d, B, max_pages;
  Cache(Operands &o, PyObject *kx, PyObject *vx, PyObject *tx, PyObject *lx, bool layered) {
    k = o.take(kx, at::kBFloat16, 4, layered ? 5 : 4);
    v = o.take(vx, at::kBFloat16, 4, layered ? 5 : 4);
    table = o.take(tx, at::kInt, 2, 2);
    lens = o.take(lx, at::kInt, 1, 1);
    if (!o.ok) return;
    if (v->sizes() != k->sizes() || lens->size(0) != table->size(0)) {
      o.fail();
      return;
    }
    const int64_t r = k->dim() - 4;
    if (r == 1) layers = size(k, 0);
    num_pages = size(k, r);
    page_size = size(k, r + 1);
    Hkv = size(k, r + 2);
    d = size(k, r + 3);
    B = size(table, 0);
    max_pages = size(table, 1);
  }
};

// A call's workspace, from torch's allocator on the current stream: given back when
// the call has been enqueued, reused only by later work on that stream.
struct Workspace {
  const size_t bytes;
  void *const p;
  explicit Workspace(size_t n) : bytes(n), p(c10::cuda::CUDACachingAllocator::raw_alloc(n ? n : 1)) {}
  ~Workspace() { c10::cuda::CUDACachingAllocator::raw_delete(p); }
  Workspace(const Workspace &) = delete;
};

PyObject *status_or(int status, PyObject *result) {
  if (status == FA_OK) return result;
  Py_XDECREF(result);
  return PyLong_FromLong(status);
}

// cache_append(k, v, k_pages, v_pages, page_table, cache_lens, cu_seqlens)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) Py_RETURN_NONE;
  Operands o;
  const Cache c(o, a[2], a[3], a[4], a[5], false);
  const at::Tensor *k = o.take(a[0], at::kBFloat16, 3, 3), *v = o.take(a[1], at::kBFloat16, 3, 3);
  const at::Tensor *cu = o.take(a[6], at::kInt, 1, 1);
  if (!o.current() || k->size(1) != c.Hkv || k->size(2) != c.d || v->sizes() != k->sizes() || cu->size(0) != (int64_t)c.B + 1)
    Py_RETURN_NONE;
  const int total = size(k, 0);
  if (total == 0) return PyLong_FromLong(FA_OK);
  return PyLong_FromLong(g_append(k->data_ptr(), v->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), ints(c.table), ints(c.lens),
                                  ints(cu), c.B, c.max_pages, c.num_pages, c.page_size, total, c.Hkv, c.d, o.stream()));
  END_HANDLE_TH_ERRORS
}

// attention_fwd_paged(q, k_pages, v_pages, page_table, cache_lens, cu_seqlens, max_new, tree_mask, scale) -> (o, lse)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || !PyLong_CheckExact(a[6]) || !(a[8] == Py_None || PyFloat_CheckExact(a[8]))) Py_RETURN_NONE;
  int overflow = 0;
  const long max_new = PyLong_AsLongAndOverflow(a[6], &overflow);
  if (overflow || max_new <= 0 || max_new > INT_MAX) Py_RETURN_NONE;
  Operands o;
  const Cache c(o, a[1], a[2], a[3], a[4], false);
  const at::Tensor *q = o.take(a[0], at::kBFloat16, 3, 3), *cu = o.take(a[5], at::kInt, 1, 1), *mask = nullptr;
  const int words = (int)((max_new + 63) / 64);
  if (a[7] != Py_None) mask = o.take(a[7], at::kLong, 2, 2);
  if (!o.current() || q->size(2) != c.d || cu->size(0) != (int64_t)c.B + 1) Py_RETURN_NONE;
  const int total = size(q, 0), H = size(q, 1);
  if (mask && (mask->size(0) != total || mask->size(1) != words)) Py_RETURN_NONE;
  const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)c.d)) : (float)PyFloat_AS_DOUBLE(a[8]);
  const auto device = q->options();
  at::Tensor out = at::empty(q->sizes(), device), lse = at::empty({H, total}, device.dtype(at::kFloat));
  int status = FA_OK;
  if (total > 0) {
    const Workspace workspace(g_paged_bytes(c.B, (int)max_new, H, c.Hkv, c.d));
    status = g_paged(q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), ints(c.table), ints(c.lens), ints(cu),
                     mask ? static_cast<const long long *>(mask->data_ptr()) : nullptr, mask ? words : 0, out.data_ptr(),
                     static_cast<float *>(lse.data_ptr()), c.B, c.max_pages, c.num_pages, c.page_size, (int)max_new, total, H,
                     c.Hkv, c.d, scale, workspace.p, workspace.bytes, o.stream());
  }
  if (status != FA_OK) return PyLong_FromLong(status);
  PyObject *x = THPVariable_Wrap(std::move(out)), *y = THPVariable_Wrap(std::move(lse));
  PyObject *both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
  END_HANDLE_TH_ERRORS
}

// cache_compact(k_pages, v_pages, page_table, cache_lens, accepted, n_accepted) -> lens
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  Operands o;
  const Cache c(o, a[0], a[1], a[2], a[3], true);
  const at::Tensor *path = o.take(a[4], at::kInt, 2, 2), *kept = o.take(a[5], at::kInt, 1, 1);
  if (!o.current() || path->size(0) != c.B || kept->size(0) != c.B) Py_RETURN_NONE;
  if (path->size(1) == 0) return THPVariable_Wrap(c.lens->clone());  // no path has a token
  at::Tensor lens = at::empty({c.B}, c.lens->options());
  const int status = g_compact(c.k->data_ptr(), c.v->data_ptr(), ints(c.table), ints(c.lens), ints(path), ints(kept),
                               ints(&lens), c.B, size(path, 1), c.max_pages, c.num_pages, c.page_size, c.layers, c.Hkv, c.d,
                               o.stream());
  return status_or(status, THPVariable_Wrap(std::move(lens)));
  END_HANDLE_TH_ERRORS
}

// cache_fork(page_refs, page_table, cache_lens, parents, page_size) -> lens
PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !PyLong_CheckExact(a[4])) Py_RETURN_NONE;
  int overflow = 0;
  const long page_size = PyLong_AsLongAndOverflow(a[4], &overflow);
  if (overflow || page_size < INT_MIN || page_size > INT_MAX) Py_RETURN_NONE;
  Operands o;
  const at::Tensor *refs = o.take(a[0], at::kInt, 1, 1), *table = o.take(a[1], at::kInt, 2, 2);
  const at::Tensor *had = o.take(a[2], at::kInt, 1, 1), *parents = o.take(a[3], at::kInt, 1, 1);
  if (!o.current() || had->size(0) != table->size(0) || parents->size(0) != table->size(0)) Py_RETURN_NONE;
  at::Tensor lens = at::empty(had->sizes(), had->options());
  const int status = g_fork(ints(refs), ints(table), ints(had), ints(parents), ints(&lens), size(table, 0), size(table, 1),
                            size(refs, 0), (int)page_size, o.stream());
  return status_or(status, THPVariable_Wrap(std::move(lens)));
  END_HANDLE_TH_ERRORS
}

// cache_resize(page_refs, k_pages, v_pages, page_table, cache_lens, new_lens) -> (lens, status)
PyObject *resize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  Operands o;
  const Cache c(o, a[1], a[2], a[3], a[4], true);
  const at::Tensor *refs = o.take(a[0], at::kInt, 1, 1), *want = o.take(a[5], at::kInt, 1, 1);
  if (!o.current() || refs->size(0) != c.num_pages || want->size(0) != c.B) Py_RETURN_NONE;
  at::Tensor lens = at::empty({c.B}, c.lens->options()), said = at::empty({2}, c.lens->options());
  const Workspace workspace(g_resize_bytes(c.B));
  const int status = g_resize(ints(refs), c.k->data_ptr(), c.v->data_ptr(), ints(c.table), ints(c.lens), ints(want),
                              ints(&lens), ints(&said), c.B, c.max_pages, c.num_pages, c.page_size, c.layers, c.Hkv, c.d,
                              workspace.p, workspace.bytes, o.stream());
  if (status != FA_OK) return PyLong_FromLong(status);
  PyObject *x = THPVariable_Wrap(std::move(lens)), *y = THPVariable_Wrap(std::move(said));
  PyObject *both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
  END_HANDLE_TH_ERRORS
}

// connect(addresses of the C entry points, in the order of the pointers above)
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *f[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "connect takes the addresses of 7 entry points");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_paged_bytes = reinterpret_cast<decltype(g_paged_bytes)>(f[1]);
  g_paged = reinterpret_cast<decltype(g_paged)>(f[2]);
  g_compact = reinterpret_cast<decltype(g_compact)>(f[3]);
  g_fork = reinterpret_cast<decltype(g_fork)>(f[4]);
  g_resize_bytes = reinterpret_cast<decltype(g_resize_bytes)>(f[5]);
  g_resize = reinterpret_cast<decltype(g_resize)>(f[6]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(connect)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(attention)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(compact)), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(fork)), METH_FASTCALL, nullptr},
    {"resize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(resize)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
