// paged_calls.cpp - the paged calls of the Python binding, their argument checks in one native pass.
// They run once per generated token and cost a host more than the GPU where a batch is small: checked
// one attribute at a time from Python, a call takes 9-10 us on the host, here 4-5 with the launch (one row
// range read back 9.4 -> 4.1, attention of one sequence 9.9 -> 5.4).
//
// Each function returns the status of the C call, or None where the arguments are anything but plain
// (another type, shape, device or stride than expected, another device current): the binding's own
// checks then say what is wrong, or make the call. Nothing is kept between calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>

#include "quail.h"

namespace {

using at::ScalarType;

PyTypeObject* desc_type = nullptr;  // the binding's PagedDesc
decltype(&quail_paged_kv_append) append_fn = nullptr;
decltype(&quail_paged_kv_read) read_fn = nullptr;
decltype(&quail_paged_decode_attn) decode_fn = nullptr;
decltype(&quail_paged_kv_evict) evict_fn = nullptr;

// The checks of one call; `ok` falls with the first that fails. Addresses are taken as the binding's own
// checks take them, for writing: a tensor that shares its memory with a lazy clone gets its own first
// (inputs too: an eviction may name one pool as both).
struct Call {
  quail_paged_desc d{};
  int index = -1;
  bool ok = false;

  explicit Call(PyObject* desc) {
    if (Py_TYPE(desc) != desc_type) return;
    Py_buffer view;
    if (PyObject_GetBuffer(desc, &view, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      return;
    }
    ok = view.len == static_cast<Py_ssize_t>(sizeof(d));
    if (ok) memcpy(&d, view.buf, sizeof(d));
    PyBuffer_Release(&view);
    index = c10::cuda::current_device();
  }
  const at::Tensor* tensor(PyObject* o, ScalarType type) {
    if (ok && THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.scalar_type() == type && t.layout() == at::kStrided && t.device().is_cuda() &&
          t.device().index() == index)
        return &t;
    }
    ok = false;
    return nullptr;
  }
  // A contiguous tensor of exactly this shape; None is NULL where it may be.
  void* exact(PyObject* o, ScalarType type, at::IntArrayRef shape, bool none = false) {
    if (none && o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o, type);
    if (t == nullptr) return nullptr;
    ok = t->sizes() == shape && t->is_contiguous();
    return ok ? t->mutable_data_ptr() : nullptr;
  }
  // bf16 rows [n, heads, d] any distance apart; n < 0: as many as there are.
  void* rows(PyObject* o, int64_t& n, int64_t heads, int64_t& stride) {
    const at::Tensor* t = tensor(o, ScalarType::BFloat16);
    if (t == nullptr) return nullptr;
    const int64_t width = d.head_dim;
    ok = t->dim() == 3 && (n < 0 || t->size(0) == n) && t->size(1) == heads && t->size(2) == width;
    if (!ok) return nullptr;
    n = t->size(0);
    ok = n == 0 || (t->stride(2) == 1 && (t->stride(1) == width || heads <= 1));
    stride = n > 1 ? t->stride(0) : heads * width;
    return ok ? t->mutable_data_ptr() : nullptr;
  }
  void* pool(PyObject* o, int64_t pages) {
    const int64_t hkv = d.num_kv_heads, page = d.page_size, width = d.head_dim;
    if (d.kv_dtype == QUAIL_FP4_E2M1) return exact(o, ScalarType::Byte, {pages, hkv, page * width * 9 / 16});
    ScalarType type = ScalarType::BFloat16;
    if (d.kv_dtype == QUAIL_FP8_E4M3)
      type = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == ScalarType::Byte
                 ? ScalarType::Byte : ScalarType::Float8_e4m3fn;
    return exact(o, type, {pages, page, hkv, width});
  }
  void pools(PyObject* k, PyObject* v, int64_t pages, void*& kp, void*& vp) {
    kp = pool(k, pages);
    vp = pool(v, pages);
    if (ok) ok = THPVariable_Unpack(k).scalar_type() == THPVariable_Unpack(v).scalar_type();
  }
  void scales(PyObject* k, PyObject* v, float*& ks, float*& vs) {
    ks = vs = nullptr;
    if (d.kv_dtype == QUAIL_BF16) {
      ok = ok && k == Py_None && v == Py_None;
      return;
    }
    ks = static_cast<float*>(exact(k, ScalarType::Float, {d.num_seqs, d.num_kv_heads}));
    vs = static_cast<float*>(exact(v, ScalarType::Float, {d.num_seqs, d.num_kv_heads}));
  }
  int32_t* ints(PyObject* o, at::IntArrayRef shape, bool none = false) {
    return static_cast<int32_t*>(exact(o, ScalarType::Int, shape, none));
  }
  int32_t* table(PyObject* o) { return ints(o, {d.num_seqs, d.max_pages_per_seq}); }
  // [B, Hkv, n] fp32, n >= least
  float* score(PyObject* o, int64_t least, int64_t& width) {
    const at::Tensor* t = tensor(o, ScalarType::Float);
    if (t == nullptr) return nullptr;
    ok = t->dim() == 3 && t->size(0) == d.num_seqs && t->size(1) == d.num_kv_heads &&
         t->size(2) >= least && t->is_contiguous();
    if (!ok) return nullptr;
    width = t->size(2);
    return static_cast<float*>(t->mutable_data_ptr());
  }
  void* workspace(PyObject* o, size_t& bytes) {
    const at::Tensor* t = tensor(o, ScalarType::Byte);
    if (t == nullptr) return nullptr;
    ok = t->dim() == 1 && t->is_contiguous();
    bytes = static_cast<size_t>(t->numel());
    return ok ? t->mutable_data_ptr() : nullptr;
  }
  int32_t number(PyObject* o) {  // of a non-negative 32-bit value
    if (!PyLong_CheckExact(o)) {
      ok = false;
      return 0;
    }
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) PyErr_Clear();
    ok = ok && x >= 0 && x <= INT32_MAX;
    return ok ? static_cast<int32_t>(x) : 0;
  }
  template <class F>
  PyObject* done(F&& fn) {
    if (!ok) Py_RETURN_NONE;
    quail_stream_t stream = reinterpret_cast<quail_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
    quail_status status;
    Py_BEGIN_ALLOW_THREADS;
    status = fn(stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
  }
};

// (desc, k_new, v_new, start_pos, block_table, k_pages, v_pages, new_offsets, k_scale, v_scale)
PyObject* call_append(PyObject*, PyObject* const* v, Py_ssize_t count) try {
  if (count != 10 || append_fn == nullptr) Py_RETURN_NONE;
  Call c(v[0]);
  int64_t n = -1, ks = 0, vs = 0;
  void *k = c.rows(v[1], n, c.d.num_kv_heads, ks), *w = c.rows(v[2], n, c.d.num_kv_heads, vs);
  int32_t *start = c.ints(v[3], {c.d.num_seqs}), *table = c.table(v[4]);
  void *kp, *vp;
  c.pools(v[5], v[6], c.d.num_pages, kp, vp);
  int32_t* off = c.ints(v[7], {static_cast<int64_t>(c.d.num_seqs) + 1}, true);
  float *sk, *sv;
  c.scales(v[8], v[9], sk, sv);
  return c.done([&](quail_stream_t s) {
    return append_fn(&c.d, n, k, w, ks, vs, off, start, table, sk, sv, kp, vp, s);
  });
} catch (...) {
  Py_RETURN_NONE;
}

// (desc, k_pages, v_pages, start_pos, block_table, k_out, v_out, offsets, k_scale, v_scale)
PyObject* call_read(PyObject*, PyObject* const* v, Py_ssize_t count) try {
  if (count != 10 || read_fn == nullptr || v[5] == Py_None || v[6] == Py_None) Py_RETURN_NONE;
  Call c(v[0]);
  int64_t n = -1, ks = 0, vs = 0;
  void *k = c.rows(v[5], n, c.d.num_kv_heads, ks), *w = c.rows(v[6], n, c.d.num_kv_heads, vs);
  int32_t *start = c.ints(v[3], {c.d.num_seqs}), *table = c.table(v[4]);
  void *kp, *vp;
  c.pools(v[1], v[2], c.d.num_pages, kp, vp);
  int32_t* off = c.ints(v[7], {static_cast<int64_t>(c.d.num_seqs) + 1}, true);
  float *sk, *sv;
  c.scales(v[8], v[9], sk, sv);
  return c.done([&](quail_stream_t s) {
    return read_fn(&c.d, n, off, start, table, sk, sv, kp, vp, k, w, ks, vs, s);
  });
} catch (...) {
  Py_RETURN_NONE;
}

// (desc, q, k_pages, v_pages, block_table, seq_lens, out, workspace, lse, k_scale, v_scale, score_in,
//  score_out)
PyObject* call_decode(PyObject*, PyObject* const* v, Py_ssize_t count) try {
  if (count != 13 || decode_fn == nullptr) Py_RETURN_NONE;
  Call c(v[0]);
  const int64_t hq = c.d.num_q_heads;
  int64_t n = c.d.num_seqs, stride = 0, width = 0;
  void* q = c.rows(v[1], n, hq, stride);
  void *kp, *vp;
  c.pools(v[2], v[3], c.d.num_pages, kp, vp);
  int32_t *table = c.table(v[4]), *lens = c.ints(v[5], {n});
  void* out = c.exact(v[6], ScalarType::BFloat16, {n, hq, c.d.head_dim});
  size_t bytes = 0;
  void* ws = c.workspace(v[7], bytes);
  float* lse = static_cast<float*>(c.exact(v[8], ScalarType::Float, {n, hq}, true));
  float *sk, *sv, *in = nullptr, *sum = nullptr;
  c.scales(v[9], v[10], sk, sv);
  if (v[12] != Py_None) {
    sum = c.score(v[12], c.d.max_seq_len, width);
    in = static_cast<float*>(c.exact(v[11], ScalarType::Float, {n, c.d.num_kv_heads, width}, true));
  } else if (v[11] != Py_None) {
    Py_RETURN_NONE;
  }
  return c.done([&](quail_stream_t s) {
    return decode_fn(&c.d, q, stride, kp, vp, table, lens, sk, sv, out, lse, in, sum, width, ws, bytes, s);
  });
} catch (...) {
  Py_RETURN_NONE;
}

// (desc, budget, recent, k_pages, v_pages, block_table, seq_lens, score, dst_table, k_dst, v_dst, kept,
//  new_lens, workspace, score_out)
PyObject* call_evict(PyObject*, PyObject* const* v, Py_ssize_t count) try {
  if (count != 15 || evict_fn == nullptr) Py_RETURN_NONE;
  Call c(v[0]);
  const int32_t budget = c.number(v[1]), recent = c.number(v[2]);
  void *kp, *vp, *kd, *vd;
  c.pools(v[3], v[4], c.d.num_pages, kp, vp);
  int32_t *table = c.table(v[5]), *lens = c.ints(v[6], {c.d.num_seqs});
  int64_t width = 0, out_width = 0, dst_pages = 0, dst_width = 0;
  float* score = c.score(v[7], c.d.max_seq_len, width);
  const at::Tensor* dst = c.tensor(v[8], ScalarType::Int);
  if (dst != nullptr) {
    c.ok = dst->dim() == 2 && dst->size(1) <= INT32_MAX;
    if (c.ok) dst_width = dst->size(1);
  }
  if (c.ok && THPVariable_Check(v[9]) && THPVariable_Unpack(v[9]).dim() > 0)
    dst_pages = THPVariable_Unpack(v[9]).size(0);
  if (dst_pages > INT32_MAX) Py_RETURN_NONE;
  int32_t* to = c.ints(v[8], {c.d.num_seqs, dst_width});
  c.pools(v[9], v[10], dst_pages, kd, vd);
  int32_t* kept = c.ints(v[11], {c.d.num_seqs, c.d.num_kv_heads, budget});
  int32_t* fresh = c.ints(v[12], {c.d.num_seqs});
  size_t bytes = 0;
  void* ws = c.workspace(v[13], bytes);
  float* out = v[14] == Py_None ? nullptr : c.score(v[14], budget, out_width);
  return c.done([&](quail_stream_t s) {
    return evict_fn(&c.d, budget, recent, kp, vp, table, lens, score, width, to,
                    static_cast<int32_t>(dst_width), static_cast<int32_t>(dst_pages), kd, vd, kept, fresh,
                    out, out_width, ws, bytes, s);
  });
} catch (...) {
  Py_RETURN_NONE;
}

// (PagedDesc, addresses of the four entry points of the loaded library)
PyObject* call_bind(PyObject*, PyObject* const* v, Py_ssize_t count) {
  if (count != 5 || !PyType_Check(v[0])) {
    PyErr_SetString(PyExc_TypeError, "bind(type, append, read, decode, evict)");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(v[1 + i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: an address is NULL");
      return nullptr;
    }
  }
  Py_INCREF(v[0]);
  desc_type = reinterpret_cast<PyTypeObject*>(v[0]);
  append_fn = reinterpret_cast<decltype(append_fn)>(p[0]);
  read_fn = reinterpret_cast<decltype(read_fn)>(p[1]);
  decode_fn = reinterpret_cast<decltype(decode_fn)>(p[2]);
  evict_fn = reinterpret_cast<decltype(evict_fn)>(p[3]);
  Py_RETURN_NONE;
}

}  // namespace

extern "C" PyObject* PyInit__paged_calls() {
  static PyMethodDef methods[] = {
      {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_bind)), METH_FASTCALL, nullptr},
      {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_append)), METH_FASTCALL, nullptr},
      {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_read)), METH_FASTCALL, nullptr},
      {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_decode)), METH_FASTCALL, nullptr},
      {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_evict)), METH_FASTCALL, nullptr},
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_calls", nullptr, -1, methods};
  return PyModule_Create(&module);
}
