// paged_binding.cpp — CPython entry points of the torch helpers around the paged cache for
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
decltype(&fa_qk_norm_rope) g_rope;
decltype(&fa_qk_norm_rope_bwd_workspace_bytes) g_rope_bytes;
decltype(&fa_qk_norm_rope_bwd) g_rope_bwd;
decltype(&fa_cache_append_rope) g_append_rope;
decltype(&fa_attention_weights_paged) g_weights;
decltype(&fa_cache_evict) g_evict;

// Rows of heads with strides, in elements (bf16 [total, heads, d] or [B, N, heads, d]).
struct HeadRows {
  const at::Tensor *x = nullptr;
  int64_t token = 0, head = 0;
  const void *data() const { return x ? x->data_ptr() : nullptr; }
};

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
  // dense heads, one stride for all tokens
  HeadRows rows(PyObject *x) {
    HeadRows r;
    if (!ok || !THPVariable_Check(x)) {
      fail();
      return r;
    }
    const at::Tensor &t = THPVariable_Unpack(x);
    const int64_t n = t.dim();
    if (!t.is_cuda() || t.scalar_type() != at::kBFloat16 || n < 3 || n > 4 || t.layout() != at::kStrided || t.numel() == 0 ||
        t.numel() / (t.size(n - 2) * t.size(n - 1)) > INT_MAX || t.size(n - 2) > INT_MAX || t.size(n - 1) > INT_MAX) {
      fail();
      return r;
    }
    if (device < 0) device = t.get_device();
    r.token = t.stride(n - 3);
    if (n == 4 && t.size(0) > 1) {
      if (t.size(1) == 1) r.token = t.stride(0);
      else if (t.stride(0) != t.size(1) * r.token) fail();
    }
    if (t.get_device() != device || t.stride(n - 1) != 1) fail();
    if (t.numel() == t.size(n - 2) * t.size(n - 1)) r.token = 0;
    r.head = t.size(n - 2) == 1 ? 0 : t.stride(n - 2);
    r.x = &t;
    return r;
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

bool same_lead(const at::Tensor *a, const at::Tensor *b) {  // tokens and d
  if (a->dim() != b->dim() || a->size(-1) != b->size(-1)) return false;
  for (int64_t i = 0; i + 2 < a->dim(); ++i)
    if (a->size(i) != b->size(i)) return false;
  return true;
}

bool number(PyObject *x, int *to) {
  if (!PyLong_CheckExact(x)) return false;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(x, &overflow);
  if (overflow || v < INT_MIN || v > INT_MAX) return false;
  *to = (int)v;
  return true;
}

// positions, inv_freq, the weights of the norms, eps, axes, interleaved
struct Turning {
  const at::Tensor *positions = nullptr, *inv_freq, *wq = nullptr, *wk = nullptr;
  int n_axes = 1, rot = 0, axis[128];
  const int *axes = nullptr;
  int bf16 = 0, interleaved = 0;
  float eps = 0;
  // lead: the dimensions of q before its heads
  Turning(Operands &o, const at::Tensor *q, PyObject *px, PyObject *fx, PyObject *wqx, PyObject *wkx, PyObject *ex,
          PyObject *ax, PyObject *ix) {
    inv_freq = o.take(fx, at::kFloat, 1, 1);
    if (!o.ok || !PyFloat_CheckExact(ex) || !PyBool_Check(ix)) {
      o.fail();
      return;
    }
    eps = (float)PyFloat_AS_DOUBLE(ex);
    interleaved = ix == Py_True;
    const int64_t half = inv_freq->size(0), lead = q->dim() - 2;
    rot = (int)(2 * half);
    if (px != Py_None) {
      positions = o.take(px, at::kInt, lead, lead + 1);
      if (!o.ok) return;
      const int64_t extra = positions->dim() - lead;
      if (extra != (ax != Py_None)) o.fail();
      for (int64_t i = 0; i < lead; ++i)
        if (positions->size(extra + i) != q->size(i)) o.fail();
      if (extra) n_axes = size(positions, 0);
    }
    if (ax != Py_None) {
      if (!PyTuple_CheckExact(ax) || half > 128 || PyTuple_GET_SIZE(ax) != half) {
        o.fail();
        return;
      }
      int most = 0;
      for (int64_t i = 0; i < half; ++i) {
        if (!number(PyTuple_GET_ITEM(ax, i), &axis[i]) || axis[i] < 0) {
          o.fail();
          return;
        }
        if (axis[i] > most) most = axis[i];
      }
      if (!positions) n_axes = most + 1;
      if (most >= n_axes) o.fail();
      axes = axis;
    }
    auto weight = [&](PyObject *x) -> const at::Tensor * {
      if (x == Py_None || !o.ok) return nullptr;
      const bool b = THPVariable_Check(x) && THPVariable_Unpack(x).scalar_type() == at::kBFloat16;
      const at::Tensor *w = o.take(x, b ? at::kBFloat16 : at::kFloat, 1, 1);
      if (!o.ok || w->size(0) != q->size(-1) || (wq && bf16 != b)) return o.fail();
      bf16 = b;
      return w;
    };
    wq = weight(wqx);
    wk = weight(wkx);
  }
  const int *at() const { return positions ? ints(positions) : nullptr; }
  const float *freq() const { return static_cast<const float *>(inv_freq->data_ptr()); }
  static const void *data(const at::Tensor *w) { return w ? w->data_ptr() : nullptr; }
};

int tokens_of(const at::Tensor *q) { return (int)(q->numel() / (q->size(-2) * q->size(-1))); }
PyObject *pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  PyObject *both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
}

// qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, axes, interleaved) -> (q, k)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || a[2] == Py_None) Py_RETURN_NONE;
  Operands o;
  const HeadRows q = o.rows(a[0]), k = o.rows(a[1]);
  if (!o.ok || !same_lead(q.x, k.x)) Py_RETURN_NONE;
  const Turning r(o, q.x, a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
  if (!o.current()) Py_RETURN_NONE;
  at::Tensor qo = at::empty(q.x->sizes(), q.x->options()), ko = at::empty(k.x->sizes(), k.x->options());
  const int status = g_rope(q.data(), q.token, q.head, k.data(), k.token, k.head, r.at(), r.n_axes, r.freq(), r.rot, r.axes,
                            r.data(r.wq), r.data(r.wk), r.bf16, r.eps, r.interleaved, qo.data_ptr(), ko.data_ptr(),
                            tokens_of(q.x), size(q.x, -2), size(k.x, -2), size(q.x, -1), o.stream());
  if (status != FA_OK) return PyLong_FromLong(status);
  return pair(std::move(qo), std::move(ko));
  END_HANDLE_TH_ERRORS
}

// qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight, eps, axes, interleaved)
//   -> (dq, dk, dq_weight, dk_weight)
PyObject *rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11 || a[4] == Py_None) Py_RETURN_NONE;
  Operands o;
  const HeadRows gq = o.rows(a[0]), gk = o.rows(a[1]);
  if (!o.ok || !same_lead(gq.x, gk.x)) Py_RETURN_NONE;
  const Turning r(o, gq.x, a[4], a[5], a[6], a[7], a[8], a[9], a[10]);
  HeadRows q, k;
  if (o.ok && r.wq) q = o.rows(a[2]);
  if (o.ok && r.wk) k = o.rows(a[3]);
  if (!o.current() || (q.x && q.x->sizes() != gq.x->sizes()) || (k.x && k.x->sizes() != gk.x->sizes())) Py_RETURN_NONE;
  const int d = size(gq.x, -1);
  at::Tensor dq = at::empty(gq.x->sizes(), gq.x->options()), dk = at::empty(gk.x->sizes(), gk.x->options()), dwq, dwk;
  const auto sums = gq.x->options().dtype(at::kFloat);
  if (r.wq) dwq = at::empty({d}, sums);
  if (r.wk) dwk = at::empty({d}, sums);
  auto floats = [](const at::Tensor &t) { return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr; };
  const Workspace workspace(r.wq || r.wk ? g_rope_bytes(d) : 0);
  const int status = g_rope_bwd(gq.data(), gq.token, gq.head, gk.data(), gk.token, gk.head, q.data(), q.token, q.head, k.data(),
                                k.token, k.head, r.at(), r.n_axes, r.freq(), r.rot, r.axes, r.data(r.wq), r.data(r.wk), r.bf16,
                                r.eps, r.interleaved, dq.data_ptr(), dk.data_ptr(), floats(dwq), floats(dwk), tokens_of(gq.x),
                                size(gq.x, -2), size(gk.x, -2), d, workspace.p, workspace.bytes, o.stream());
  if (status != FA_OK) return PyLong_FromLong(status);
  PyObject *all[4];
  bool good = true;
  at::Tensor *from[4] = {&dq, &dk, &dwq, &dwk};
  for (int i = 0; i < 4; ++i) {
    if (from[i]->defined()) {
      all[i] = THPVariable_Wrap(std::move(*from[i]));
    } else {
      all[i] = Py_None;
      Py_INCREF(Py_None);
    }
    good &= all[i] != nullptr;
  }
  PyObject *four = good ? PyTuple_Pack(4, all[0], all[1], all[2], all[3]) : nullptr;
  for (PyObject *x : all) Py_XDECREF(x);
  return four;
  END_HANDLE_TH_ERRORS
}

// cache_append_rope(q, k, v, k_pages, v_pages, page_table, cache_lens, cu_seqlens, inv_freq, positions, q_weight,
//                   k_weight, eps, axes, interleaved) -> q
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) Py_RETURN_NONE;
  Operands o;
  const Cache c(o, a[3], a[4], a[5], a[6], false);
  const at::Tensor *cu = o.take(a[7], at::kInt, 1, 1);
  const HeadRows q = o.rows(a[0]), k = o.rows(a[1]), v = o.rows(a[2]);
  if (!o.ok || q.x->dim() != 3 || !same_lead(q.x, k.x) || v.x->sizes() != k.x->sizes() || k.x->size(1) != c.Hkv ||
      k.x->size(2) != c.d || cu->size(0) != (int64_t)c.B + 1)
    Py_RETURN_NONE;
  const Turning r(o, q.x, a[9], a[8], a[10], a[11], a[12], a[13], a[14]);
  if (!o.current()) Py_RETURN_NONE;
  at::Tensor qo = at::empty(q.x->sizes(), q.x->options());
  const int status = g_append_rope(q.data(), q.token, q.head, k.data(), k.token, k.head, v.data(), v.token, v.head,
                                   c.k->data_ptr(), c.v->data_ptr(), ints(c.table), ints(c.lens), ints(cu), r.at(), r.n_axes,
                                   r.freq(), r.rot, r.axes, r.data(r.wq), r.data(r.wk), r.bf16, r.eps, r.interleaved,
                                   qo.data_ptr(), c.B, c.max_pages, c.num_pages, c.page_size, tokens_of(q.x), size(q.x, 1),
                                   c.Hkv, c.d, o.stream());
  return status_or(status, THPVariable_Wrap(std::move(qo)));
  END_HANDLE_TH_ERRORS
}

// attention_weights_paged(q, k_pages, page_table, cache_lens, cu_seqlens, max_new, lse, weights, tree_mask, decay, scale)
//   -> status
PyObject *weights(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int max_new = 0;
  if (n != 11 || !number(a[5], &max_new) || max_new <= 0 || !PyFloat_CheckExact(a[9]) ||
      !(a[10] == Py_None || PyFloat_CheckExact(a[10])))
    Py_RETURN_NONE;
  Operands o;
  const Cache c(o, a[1], a[1], a[2], a[3], false);
  const at::Tensor *q = o.take(a[0], at::kBFloat16, 3, 3), *cu = o.take(a[4], at::kInt, 1, 1);
  const at::Tensor *lse = o.take(a[6], at::kFloat, 2, 2), *w = o.take(a[7], at::kFloat, 3, 3), *mask = nullptr;
  if (a[8] != Py_None) mask = o.take(a[8], at::kLong, 2, 2);
  if (!o.current() || q->size(2) != c.d || cu->size(0) != (int64_t)c.B + 1) Py_RETURN_NONE;
  const int total = size(q, 0), H = size(q, 1), words = (int)(((int64_t)max_new + 63) / 64);
  if ((mask && (mask->size(0) != total || mask->size(1) != words)) || lse->size(0) != H || lse->size(1) != total ||
      w->size(0) != c.B || w->size(1) != c.Hkv)
    Py_RETURN_NONE;
  const float scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)c.d)) : (float)PyFloat_AS_DOUBLE(a[10]);
  if (total == 0) return PyLong_FromLong(FA_OK);
  return PyLong_FromLong(g_weights(q->data_ptr(), c.k->data_ptr(), ints(c.table), ints(c.lens), ints(cu),
                                   mask ? static_cast<const long long *>(mask->data_ptr()) : nullptr, mask ? words : 0,
                                   static_cast<const float *>(lse->data_ptr()), static_cast<float *>(w->data_ptr()), size(w, 2),
                                   (float)PyFloat_AS_DOUBLE(a[9]), c.B, c.max_pages, c.num_pages, c.page_size, max_new, total, H,
                                   c.Hkv, c.d, scale, o.stream()));
  END_HANDLE_TH_ERRORS
}

// cache_evict(page_refs, k_pages, v_pages, page_table, cache_lens, weights, keep, recent) -> (lens, kept)
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int keep, recent;
  if (n != 8 || !number(a[6], &keep) || !number(a[7], &recent) || recent < 0 || recent > keep) Py_RETURN_NONE;
  Operands o;
  const at::Tensor *refs = o.take(a[0], at::kInt, 1, 1);
  const Cache c(o, a[1], a[2], a[3], a[4], true);
  const at::Tensor *w = o.take(a[5], at::kFloat, 3, 4);
  if (!o.current() || refs->size(0) != c.num_pages || w->dim() != c.k->dim() - 1) Py_RETURN_NONE;
  const int64_t r = w->dim() - 3;
  if ((r && w->size(0) != c.layers) || w->size(r) != c.B || w->size(r + 1) != c.Hkv) Py_RETURN_NONE;
  at::Tensor lens = at::empty({c.B}, c.lens->options());
  at::Tensor kept = r ? at::empty({c.layers, c.B, c.Hkv, keep}, c.lens->options()) : at::empty({c.B, c.Hkv, keep}, c.lens->options());
  const int status = g_evict(ints(refs), c.k->data_ptr(), c.v->data_ptr(), ints(c.table), ints(c.lens),
                             static_cast<float *>(w->data_ptr()), size(w, r + 2), keep, recent, ints(&lens), ints(&kept), c.B,
                             c.max_pages, c.num_pages, c.page_size, c.layers, c.Hkv, c.d, o.stream());
  if (status != FA_OK) return PyLong_FromLong(status);
  return pair(std::move(lens), std::move(kept));
  END_HANDLE_TH_ERRORS
}

// connect(addresses of the C entry points, in the order of the pointers above)
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *f[13];
  if (n != 13) {
    PyErr_SetString(PyExc_TypeError, "connect takes the addresses of 13 entry points");
    return nullptr;
  }
  for (int i = 0; i < 13; ++i) {
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
  g_rope = reinterpret_cast<decltype(g_rope)>(f[7]);
  g_rope_bytes = reinterpret_cast<decltype(g_rope_bytes)>(f[8]);
  g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(f[9]);
  g_append_rope = reinterpret_cast<decltype(g_append_rope)>(f[10]);
  g_weights = reinterpret_cast<decltype(g_weights)>(f[11]);
  g_evict = reinterpret_cast<decltype(g_evict)>(f[12]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(connect)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(attention)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(compact)), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(fork)), METH_FASTCALL, nullptr},
    {"resize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(resize)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope)), METH_FASTCALL, nullptr},
    {"rope_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope_bwd)), METH_FASTCALL, nullptr},
    {"append_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append_rope)), METH_FASTCALL, nullptr},
    {"weights", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(weights)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
