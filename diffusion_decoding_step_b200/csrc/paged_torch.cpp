// Python binding of the paged cache calls: takes torch tensors, checks them, and
// passes their addresses and strides to the C ABI.  The same work in Python took
// 8 of a call's 11 us on the host, three times what the append of a token takes on the
// GPU; a call takes 4 to 6 us with it.
//
// The library's functions come as addresses, so that this module needs no
// particular library file.
#include <Python.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dllm.h"

namespace {

struct Handle {
  dllm_kv_pages kv;
  at::Tensor k_pages, v_pages;
  int n_q_heads, max_rows, max_groups, index;
  at::ScalarType type;
  void* ws;
  size_t ws_bytes;
  decltype(&dllm_paged_append) append;
  decltype(&dllm_paged_attn) attn;
  decltype(&dllm_shared_prefix_attn) shared;
};

const char* kName = "dllm_paged";

Handle* handle(PyObject* o) { return static_cast<Handle*>(PyCapsule_GetPointer(o, kName)); }

void destroy(PyObject* o) { delete handle(o); }

// The tensor of an argument; null with an exception set if it is none.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_ValueError, "%s: a tensor is needed, got %s", what, Py_TYPE(o)->tp_name);
  return nullptr;
}

bool refuse(const at::Tensor& t, const char* what, const char* needed) {
  std::string shape;
  for (const int64_t n : t.sizes()) shape += (shape.empty() ? "" : ", ") + std::to_string(n);
  PyErr_Format(PyExc_ValueError, "%s: %s is needed, got %s [%s] on %s", what, needed,
               c10::toString(t.scalar_type()), shape.c_str(), t.device().str().c_str());
  return false;
}

// The operators have no backward: a tensor whose gradient autograd would expect is refused.
bool no_grad(const at::Tensor& t, const char* what) {
  if (!t.requires_grad() || !at::GradMode::is_enabled()) return true;
  PyErr_Format(PyExc_ValueError,
               "%s requires a gradient, and the paged cache has no backward: call it under "
               "torch.no_grad()",
               what);
  return false;
}

// Tells autograd that a tensor is written (inference tensors have no version).
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A contiguous tensor of `type` on the pages' GPU with the given extents (-1: any).
bool plain(const Handle& h, PyObject* o, const char* what, at::ScalarType type,
           std::initializer_list<int64_t> extents, const void** out) {
  const at::Tensor* t = tensor(o, what);
  if (!t) return false;
  bool ok = t->scalar_type() == type && t->is_cuda() && t->get_device() == h.index &&
            t->dim() == (int64_t)extents.size() && t->is_contiguous();
  int64_t i = 0;
  std::string shape;
  for (const int64_t n : extents) {
    ok = ok && (n < 0 || t->size(i) == n);
    shape += (i++ ? ", " : "") + (n < 0 ? std::string("any") : std::to_string(n));
  }
  if (!ok)
    return refuse(*t, what,
                  ("a contiguous " + std::string(type == at::kInt ? "int32" : "float32") +
                   " tensor [" + shape + "] on cuda:" + std::to_string(h.index))
                      .c_str());
  *out = t->const_data_ptr();
  return true;
}

bool ints(const Handle& h, PyObject* o, const char* what, std::initializer_list<int64_t> extents,
          const int32_t** out) {
  const void* p = nullptr;
  if (!plain(h, o, what, at::kInt, extents, &p)) return false;
  *out = static_cast<const int32_t*>(p);
  return true;
}

// Rows [n_rows][heads][D] of the pages' type with contiguous heads; OUT: that are written.
template <bool OUT = false>
bool rows(const Handle& h, PyObject* o, const char* what, int64_t n_rows, int64_t heads,
          dllm_rows* out) {
  const at::Tensor* t = tensor(o, what);
  if (!t) return false;
  if (t->scalar_type() != h.type || !t->is_cuda() || t->get_device() != h.index || t->dim() != 3 ||
      t->size(0) != n_rows || t->size(1) != heads || t->size(2) != h.kv.head_dim ||
      t->stride(2) != 1)
    return refuse(*t, what,
                  ("a " + std::string(c10::toString(h.type)) + " tensor [" +
                   std::to_string(n_rows) + ", " + std::to_string(heads) + ", " +
                   std::to_string(h.kv.head_dim) + "] on cuda:" + std::to_string(h.index) +
                   " with contiguous heads")
                      .c_str());
  if (!no_grad(*t, what)) return false;
  void* data = OUT ? t->mutable_data_ptr() : const_cast<void*>(t->const_data_ptr());
  *out = dllm_rows{data, t->stride(0), t->stride(1)};
  return true;
}

bool batch(const Handle& h, PyObject* row_start, PyObject* table, int64_t n_rows,
           dllm_paged_batch* out) {
  const at::Tensor *r = tensor(row_start, "row_start"), *t = r ? tensor(table, "page_table") : r;
  if (!t) return false;
  const int64_t n = r->numel() - 1, width = t->dim() == 2 ? t->size(1) : -1;
  if (n_rows > INT32_MAX || n > INT32_MAX || width > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "sizes beyond 2^31");
    return false;
  }
  *out = dllm_paged_batch{(int32_t)n, (int32_t)n_rows, (int32_t)width, (int32_t)width, nullptr,
                          nullptr};
  return ints(h, row_start, "row_start", {n + 1}, &out->row_start) &&
         ints(h, table, "page_table", {n, -1}, &out->page_table);
}

// A call without rows has nothing to do; the C ABI has no such calls.
template <class F>
PyObject* call(const Handle& h, int64_t n_rows, F&& f) {
  dllm_status status = DLLM_OK;
  if (n_rows == 0) return PyLong_FromLong(status);
  std::string failed;
  Py_BEGIN_ALLOW_THREADS;
  try {  // no exception may pass the restoring of the thread's state
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)h.index);
    status =
        f(reinterpret_cast<dllm_stream>(c10::cuda::getCurrentCUDAStream(h.index).stream()));
  } catch (const std::exception& e) {
    failed = e.what();
    if (failed.empty()) failed = "device guard";
  }
  Py_END_ALLOW_THREADS;
  if (!failed.empty()) return PyErr_Format(PyExc_RuntimeError, "%s", failed.c_str());
  return PyLong_FromLong(status);
}

bool given(PyObject* o) { return o != Py_None; }

// A number for the C ABI, which takes fp32, where zero stands for the default: one that
// rounds to zero is refused.
bool number(PyObject* o, const char* what, float* out) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) return false;
  *out = (float)x;
  if (x == 0.0 || *out != 0.f) return true;
  PyErr_Format(PyExc_ValueError, "%s: %S is zero in 32 bits, which stands for the default", what, o);
  return false;
}

// create(pages struct address, n_q_heads, max_rows, max_groups, device, is_f16, ws, ws_bytes,
//        append, attn, shared, k_pages, v_pages)
PyObject* create(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return PyErr_Format(PyExc_TypeError, "create: 13 arguments");
  const at::Tensor *kp = tensor(a[11], "k_pages"), *vp = kp ? tensor(a[12], "v_pages") : kp;
  if (!vp) return nullptr;
  long long v[11];
  for (int i = 0; i < 11; ++i) {
    v[i] = PyLong_AsLongLong(a[i]);
    if (v[i] == -1 && PyErr_Occurred()) return nullptr;
  }
  Handle* h = new Handle;
  h->kv = *reinterpret_cast<const dllm_kv_pages*>(v[0]);
  h->k_pages = *kp;
  h->v_pages = *vp;
  h->n_q_heads = (int)v[1];
  h->max_rows = (int)v[2];
  h->max_groups = (int)v[3];
  h->index = (int)v[4];
  h->type = v[5] ? at::kHalf : at::kBFloat16;
  h->ws = reinterpret_cast<void*>(v[6]);
  h->ws_bytes = (size_t)v[7];
  h->append = reinterpret_cast<decltype(h->append)>(v[8]);
  h->attn = reinterpret_cast<decltype(h->attn)>(v[9]);
  h->shared = reinterpret_cast<decltype(h->shared)>(v[10]);
  return PyCapsule_New(h, kName, destroy);
}

// append(handle, k, v, row_start, page_table, pos, q, q_out, rope_theta, rope_shift) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) return PyErr_Format(PyExc_TypeError, "append: 10 arguments");
  const Handle* h = handle(a[0]);
  const at::Tensor* kt = h ? tensor(a[1], "k") : nullptr;
  if (!kt) return nullptr;
  const int64_t n_rows = kt->dim() ? kt->size(0) : 0;
  dllm_paged_batch bt;
  dllm_rows k, v, q, qo;
  const int32_t *pos, *shift = nullptr;
  if (!batch(*h, a[3], a[4], n_rows, &bt) || !rows(*h, a[1], "k", n_rows, h->kv.n_kv_heads, &k) ||
      !rows(*h, a[2], "v", n_rows, h->kv.n_kv_heads, &v) ||
      !ints(*h, a[5], "pos", {bt.n_seqs}, &pos))
    return nullptr;
  const bool has_q = given(a[6]);
  if (has_q && (!rows(*h, a[6], "q", n_rows, h->n_q_heads, &q) ||
                !rows<true>(*h, a[7], "q_out", n_rows, h->n_q_heads, &qo)))
    return nullptr;
  float theta;
  if (!number(a[8], "rope_theta", &theta)) return nullptr;
  if (given(a[9]) && !ints(*h, a[9], "rope_shift", {bt.n_seqs}, &shift)) return nullptr;
  if (n_rows > 0) {
    written(h->k_pages);
    written(h->v_pages);
    if (has_q) written(*tensor(a[7], "q_out"));
  }
  return call(*h, n_rows, [&](dllm_stream s) {
    return h->append(&h->kv, &bt, has_q ? h->n_q_heads : 0, has_q ? &q : nullptr, &k, &v,
                     has_q ? &qo : nullptr, pos, shift, theta,
                     static_cast<int32_t*>(h->ws), s);
  });
}

// attn(handle, q, row_start, page_table, segs, row_limit, scale, out, lse, group_start,
//      prefix_table, prefix_len) -> status; without groups the last three are None
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return PyErr_Format(PyExc_TypeError, "attn: 12 arguments");
  const Handle* h = handle(a[0]);
  const at::Tensor* qt = h ? tensor(a[1], "q") : nullptr;
  if (!qt) return nullptr;
  const int64_t n_rows = qt->dim() ? qt->size(0) : 0;
  if (n_rows > h->max_rows)
    return PyErr_Format(PyExc_ValueError, "%lld rows: this PagedKV was made for %d",
                        (long long)n_rows, h->max_rows);
  dllm_paged_batch bt;
  dllm_rows q, out;
  const int32_t *segs, *limit = nullptr;
  const void* lse = nullptr;
  if (!batch(*h, a[2], a[3], n_rows, &bt) || !rows(*h, a[1], "q", n_rows, h->n_q_heads, &q) ||
      !ints(*h, a[4], "segs", {bt.n_seqs, 2, 2}, &segs) ||
      (given(a[5]) && !ints(*h, a[5], "row_limit", {n_rows}, &limit)) ||
      !rows<true>(*h, a[7], "out", n_rows, h->n_q_heads, &out) ||
      (given(a[8]) && !plain(*h, a[8], "lse", at::kFloat, {n_rows, h->n_q_heads}, &lse)))
    return nullptr;
  const at::Tensor* lse_t = given(a[8]) ? tensor(a[8], "lse") : nullptr;
  if (lse_t && !no_grad(*lse_t, "lse")) return nullptr;
  float scale;
  if (!number(a[6], "scale", &scale)) return nullptr;
  float* lp = lse_t ? static_cast<float*>(lse_t->mutable_data_ptr()) : nullptr;
  auto outputs_written = [&]() {
    if (n_rows == 0) return;
    written(*tensor(a[7], "out"));
    if (lse_t) written(*lse_t);
  };
  if (!given(a[9])) {
    outputs_written();
    return call(*h, n_rows, [&](dllm_stream s) {
      return h->attn(&h->kv, &bt, h->n_q_heads, segs, limit, scale, &q, &out, lp, h->ws,
                     h->ws_bytes, s);
    });
  }
  const at::Tensor *gt = tensor(a[9], "group_start"), *pt = gt ? tensor(a[10], "prefix_table") : gt;
  if (!pt) return nullptr;
  const int64_t groups = gt->numel() - 1, width = pt->dim() == 2 ? pt->size(1) : -1;
  if (h->max_groups < 1)
    return PyErr_Format(PyExc_ValueError, "this PagedKV was made without prefix groups");
  if (groups > h->max_groups || width > INT32_MAX)
    return PyErr_Format(PyExc_ValueError, "%lld prefix groups: this PagedKV was made for up to %d",
                        (long long)groups, h->max_groups);
  if (groups < 1) return PyErr_Format(PyExc_ValueError, "group_start: no prefix groups");
  dllm_prefix_groups g{(int32_t)groups, (int32_t)width, (int32_t)width, nullptr, nullptr, nullptr};
  if (!ints(*h, a[9], "group_start", {groups + 1}, &g.seq_start) ||
      !ints(*h, a[10], "prefix_table", {groups, -1}, &g.page_table) ||
      !ints(*h, a[11], "prefix_len", {groups}, &g.len))
    return nullptr;
  outputs_written();
  return call(*h, n_rows, [&](dllm_stream s) {
    return h->shared(&h->kv, &bt, &g, h->n_q_heads, segs, limit, scale, &q, &out, lp, h->ws,
                     h->ws_bytes, s);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"create", reinterpret_cast<PyCFunction>(guarded<create>), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(guarded<append>), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(guarded<attn>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_torch() { return PyModule_Create(&module); }
