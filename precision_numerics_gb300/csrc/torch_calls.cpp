// Python module _attn_torch: the serving calls' way from tensors to the C ABI
// without the interpreter's share of the work.
//
// A small serving call runs about 5 us on the GPU, and its tensor checks, output
// allocations and argument conversions take three times that in Python.  Here
// each function asks the same questions of the tensors in C++, allocates the
// outputs that were not passed, and calls the C entry point of the same name.
// Where anything is not as expected it returns None and does nothing: the Python
// function of the same name then goes through its own checks, which say what is
// wrong.  A status other than ATTN_OK raises attn.AttnError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <math.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn.h"

namespace {

using at::Tensor;

// The tensor behind a Python object, or null.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool dense(const Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
  return t != nullptr && t->is_cuda() && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}
// BF16 of this shape whose rows are contiguous.
bool rows(const Tensor* t, at::IntArrayRef shape) {
  return t != nullptr && t->is_cuda() && t->scalar_type() == at::kBFloat16 && t->sizes() == shape &&
         t->stride(-1) == 1;
}
bool ints(const Tensor* t, int64_t n) { return dense(t, at::kInt, {n}); }

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

struct Cache {
  const Tensor *k, *v, *ks, *vs, *table;
  int B, pages, hk, page, d, blocks;
};
// Five objects: k_cache, v_cache, k_scale, v_scale, block_table.
bool cache_of(PyObject* const* o, Cache* c) {
  c->k = tensor(o[0]);
  c->v = tensor(o[1]);
  c->ks = tensor(o[2]);
  c->vs = tensor(o[3]);
  c->table = tensor(o[4]);
  if (c->k == nullptr || c->k->dim() != 4 || c->table == nullptr || c->table->dim() != 2) return false;
  const auto s = c->k->sizes();
  const at::IntArrayRef scales = s.slice(0, 2);
  if (!dense(c->k, at::kChar, s) || !dense(c->v, at::kChar, s) || !dense(c->ks, at::kFloat, scales) ||
      !dense(c->vs, at::kFloat, scales) || !dense(c->table, at::kInt, c->table->sizes()))
    return false;
  for (const int64_t x : {s[0], s[1], s[2], s[3], c->table->size(0), c->table->size(1)})
    if (x > INT32_MAX) return false;
  c->pages = (int)s[0], c->hk = (int)s[1], c->page = (int)s[2], c->d = (int)s[3];
  c->B = (int)c->table->size(0), c->blocks = (int)c->table->size(1);
  return true;
}

// True and *scale, or false where the object is neither None nor a float.
bool scale_of(PyObject* o, int64_t d, float* scale) {
  if (o == Py_None) {
    *scale = (float)(1.0 / sqrt((double)d));
    return true;
  }
  if (!PyFloat_Check(o)) return false;
  *scale = (float)PyFloat_AS_DOUBLE(o);
  return true;
}

// The output passed for this place if it is right, a new one for None.
bool output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const Tensor& like, Tensor* out) {
  if (o == Py_None) {
    *out = empty(shape, type, like);
    return true;
  }
  const Tensor* t = tensor(o);
  if (!dense(t, type, shape)) return false;
  *out = *t;
  return true;
}

// Both outputs, those passed or new ones.  New small ones share one allocation, since
// each turn of the allocator costs a small call 0.6 us of the host's time (with the
// shared memory size set once a decode call went from 6.3 to 5.0 us); larger ones do
// not, so that neither keeps the other's memory.
constexpr int64_t kShared = 256 * 1024;
bool outputs(PyObject* x, PyObject* y, at::IntArrayRef x_shape, at::ScalarType x_type, at::IntArrayRef y_shape,
             at::ScalarType y_type, const Tensor& like, Tensor* a, Tensor* b) {
  if (x == Py_None && y == Py_None) {
    const int64_t a_bytes = c10::multiply_integers(x_shape) * (int64_t)c10::elementSize(x_type);
    const int64_t b_bytes = c10::multiply_integers(y_shape) * (int64_t)c10::elementSize(y_type);
    const int64_t b_at = (a_bytes + 255) / 256 * 256;
    if (a_bytes > 0 && b_bytes > 0 && b_at + b_bytes <= kShared) {
      *a = empty({(b_at + b_bytes) / (int64_t)c10::elementSize(x_type)}, x_type, like);
      *b = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(a->storage()), a->key_set(),
                                                    c10::scalarTypeToTypeMeta(y_type));
      b->unsafeGetTensorImpl()->set_storage_offset(b_at / (int64_t)c10::elementSize(y_type));
      b->unsafeGetTensorImpl()->set_sizes_contiguous(y_shape);
      a->unsafeGetTensorImpl()->set_sizes_contiguous(x_shape);
      return true;
    }
  }
  return output(x, x_shape, x_type, like, a) && output(y, y_shape, y_type, like, b);
}

cudaStream_t stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// Raises attn.AttnError for this status of the entry point `name`.
PyObject* raise(const char* name, attn_status status) {
  PyObject* module = PyImport_ImportModule("precision_numerics_gb300.attn");
  if (module == nullptr) return nullptr;
  PyObject* type = PyObject_GetAttrString(module, "AttnError");
  Py_DECREF(module);
  if (type == nullptr) return nullptr;
  PyObject* error = PyObject_CallFunction(type, "sis", name, (int)status, attn_last_error());
  if (error != nullptr) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_DECREF(type);
  return nullptr;
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = x != nullptr ? THPVariable_Wrap(b) : nullptr;
  PyObject* r = y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// (q, k, v, plan, scale, causal, o, lse)
PyObject* varlen_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *plan = tensor(a[3]);
  if (q == nullptr || q->dim() != 3 || k == nullptr || k->dim() != 3 || plan == nullptr || !plan->is_cuda() ||
      !plan->is_contiguous())
    Py_RETURN_NONE;
  const int64_t T = q->size(0), H = q->size(1), d = q->size(2), hk = k->size(1);
  float scale;
  const int causal = PyObject_IsTrue(a[5]);
  if (causal < 0) return nullptr;
  if (!rows(q, q->sizes()) || !rows(k, {T, hk, d}) || !rows(v, {T, hk, d}) || H < 1 || hk < 1 || H % hk != 0 ||
      T > INT32_MAX || H > INT32_MAX || d > INT32_MAX || !scale_of(a[4], d, &scale))
    Py_RETURN_NONE;
  const int64_t bytes = (int64_t)plan->nbytes();
  const int64_t per = 128 / std::max<int64_t>(1, std::min<int64_t>(128, H / hk));
  const int64_t B = (bytes - 256) / 16 - T / per;
  Tensor o, lse;
  if (B < 1 || B > INT32_MAX ||
      !outputs(a[6], a[7], {T, H, d}, at::kBFloat16, {T, H}, at::kFloat, *q, &o, &lse))
    Py_RETURN_NONE;
  const attn_status s =
      attn_varlen_fwd(q->data_ptr(), k->data_ptr(), v->data_ptr(), q->stride(0), q->stride(1), k->stride(0),
                      k->stride(1), v->stride(0), v->stride(1), plan->data_ptr(), (size_t)bytes, o.data_ptr(),
                      (float*)lse.data_ptr(), (int)B, (int)T, (int)H, (int)hk, (int)d, scale, causal, stream());
  return s == ATTN_OK ? pair(o, lse) : raise("attn_varlen_fwd", s);
  END_HANDLE_TH_ERRORS
}

// (k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, starts, lens)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  if (n != 10 || !cache_of(a + 2, &c)) Py_RETURN_NONE;
  const Tensor *k = tensor(a[0]), *v = tensor(a[1]), *cu = tensor(a[7]), *starts = tensor(a[8]);
  if (k == nullptr || k->dim() != 3) Py_RETURN_NONE;
  const int64_t T = k->size(0);
  if (T > INT32_MAX || !rows(k, {T, c.hk, c.d}) || !rows(v, {T, c.hk, c.d}) || !ints(cu, c.B + (int64_t)1) ||
      !ints(starts, c.B))
    Py_RETURN_NONE;
  if (a[9] != Py_None) {
    const Tensor* lens = tensor(a[9]);
    if (!ints(lens, c.B)) Py_RETURN_NONE;
    const attn_status s = attn_cache_append_served_int8(
        k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), v->stride(0), v->stride(1), c.k->data_ptr(),
        c.v->data_ptr(), (float*)c.ks->data_ptr(), (float*)c.vs->data_ptr(), (const int*)c.table->data_ptr(),
        (const int*)cu->data_ptr(), (const int*)starts->data_ptr(), (const int*)lens->data_ptr(), c.B, (int)T, c.hk, c.d,
        c.pages, c.page, c.blocks, stream());
    return s == ATTN_OK ? PyTuple_Pack(2, a[2], a[3]) : raise("attn_cache_append_served_int8", s);
  }
  const attn_status s = attn_cache_append_int8(
      k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), v->stride(0), v->stride(1), c.k->data_ptr(),
      c.v->data_ptr(), (float*)c.ks->data_ptr(), (float*)c.vs->data_ptr(), (const int*)c.table->data_ptr(),
      (const int*)cu->data_ptr(), (const int*)starts->data_ptr(), c.B, (int)T, c.hk, c.d, c.pages, c.page, c.blocks,
      stream());
  return s == ATTN_OK ? PyTuple_Pack(2, a[2], a[3]) : raise("attn_cache_append_int8", s);
  END_HANDLE_TH_ERRORS
}

// (k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, starts, T, dtype, k, v)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  if (n != 11 || !cache_of(a, &c) || !PyLong_Check(a[7]) || !THPDtype_Check(a[8])) Py_RETURN_NONE;
  const Tensor *cu = tensor(a[5]), *starts = tensor(a[6]);
  const long long T = PyLong_AsLongLong(a[7]);
  if (T == -1 && PyErr_Occurred()) return nullptr;
  const at::ScalarType type = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
  if (T < 0 || T > INT32_MAX || (type != at::kBFloat16 && type != at::kFloat) || !ints(cu, c.B + (int64_t)1) ||
      !ints(starts, c.B))
    Py_RETURN_NONE;
  Tensor k, v;
  if (!outputs(a[9], a[10], {T, c.hk, c.d}, type, {T, c.hk, c.d}, type, *c.k, &k, &v)) Py_RETURN_NONE;
  const attn_status s = attn_cache_read_int8(
      c.k->data_ptr(), c.v->data_ptr(), (const float*)c.ks->data_ptr(), (const float*)c.vs->data_ptr(),
      (const int*)c.table->data_ptr(), (const int*)cu->data_ptr(), (const int*)starts->data_ptr(), k.data_ptr(),
      v.data_ptr(), c.B, (int)T, c.hk, c.d, c.pages, c.page, c.blocks,
      type == at::kFloat ? ATTN_DTYPE_FP32 : ATTN_DTYPE_BF16, stream());
  return s == ATTN_OK ? pair(k, v) : raise("attn_cache_read_int8", s);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, scale, o, lse, workspace)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  if (n != 11 || !cache_of(a + 1, &c)) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0]), *lens = tensor(a[6]);
  float scale;
  if (q == nullptr || q->dim() != 4 || !scale_of(a[7], c.d, &scale)) Py_RETURN_NONE;
  const int64_t n_q = q->size(1), H = q->size(2);
  Tensor o, lse, ws;
  if (n_q > INT32_MAX || H > INT32_MAX || !rows(q, {c.B, n_q, H, c.d}) || !ints(lens, c.B) ||
      !outputs(a[8], a[9], {c.B, n_q, H, c.d}, at::kBFloat16, {c.B, n_q, H}, at::kFloat, *q, &o, &lse))
    Py_RETURN_NONE;
  if (a[10] == Py_None) {
    const size_t need = attn_decode_int8_workspace_bytes(c.B, (int)n_q, (int)H, c.hk, c.d, c.page, c.blocks);
    ws = empty({(int64_t)std::max<size_t>(need, 1)}, at::kByte, *q);
  } else {
    const Tensor* t = tensor(a[10]);
    if (t == nullptr || !t->is_cuda() || !t->is_contiguous()) Py_RETURN_NONE;
    ws = *t;
  }
  const attn_status s = attn_decode_int8(
      q->data_ptr(), q->stride(0), q->stride(1), q->stride(2), c.k->data_ptr(), c.v->data_ptr(),
      (const float*)c.ks->data_ptr(), (const float*)c.vs->data_ptr(), (const int*)c.table->data_ptr(),
      (const int*)lens->data_ptr(), o.data_ptr(), (float*)lse.data_ptr(), c.B, (int)n_q, (int)H, c.hk, c.d, c.pages,
      c.page, c.blocks, scale, ws.data_ptr(), ws.nbytes(), stream());
  return s == ATTN_OK ? pair(o, lse) : raise("attn_decode_int8", s);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_len, block_table, seqlens, scale, o, lse, workspace)
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) Py_RETURN_NONE;
  PyObject* const five[5] = {a[1], a[2], a[3], a[4], a[7]};
  Cache c;
  if (!cache_of(five, &c)) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0]), *pre = tensor(a[5]), *len = tensor(a[6]), *lens = tensor(a[8]);
  float scale;
  if (q == nullptr || q->dim() != 4 || pre == nullptr || pre->dim() != 1 || !scale_of(a[9], c.d, &scale))
    Py_RETURN_NONE;
  const int64_t n_q = q->size(1), H = q->size(2), blocks = pre->size(0);
  Tensor o, lse, ws;
  if (n_q > INT32_MAX || H > INT32_MAX || blocks > INT32_MAX || !rows(q, {c.B, n_q, H, c.d}) || !ints(pre, blocks) ||
      !ints(len, 1) || !ints(lens, c.B) ||
      !outputs(a[10], a[11], {c.B, n_q, H, c.d}, at::kBFloat16, {c.B, n_q, H}, at::kFloat, *q, &o, &lse))
    Py_RETURN_NONE;
  if (a[12] == Py_None) {
    const size_t need = attn_decode_shared_int8_workspace_bytes(c.B, (int)n_q, (int)H, c.hk, c.d, c.page, (int)blocks,
                                                                c.blocks);
    ws = empty({(int64_t)std::max<size_t>(need, 1)}, at::kByte, *q);
  } else {
    const Tensor* t = tensor(a[12]);
    if (t == nullptr || !t->is_cuda() || !t->is_contiguous()) Py_RETURN_NONE;
    ws = *t;
  }
  const attn_status s = attn_decode_shared_int8(
      q->data_ptr(), q->stride(0), q->stride(1), q->stride(2), c.k->data_ptr(), c.v->data_ptr(),
      (const float*)c.ks->data_ptr(), (const float*)c.vs->data_ptr(), (const int*)pre->data_ptr(), (int)blocks,
      (const int*)len->data_ptr(), (const int*)c.table->data_ptr(), (const int*)lens->data_ptr(), o.data_ptr(),
      (float*)lse.data_ptr(), c.B, (int)n_q, (int)H, c.hk, c.d, c.pages, c.page, c.blocks, scale, ws.data_ptr(),
      ws.nbytes(), stream());
  return s == ATTN_OK ? pair(o, lse) : raise("attn_decode_shared_int8", s);
  END_HANDLE_TH_ERRORS
}

// (block_table, held, wanted, free_pages, n_free, page_size, T, lens, cu_seqlens, slots, positions)
PyObject* cache_reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11 || !PyLong_Check(a[5]) || !PyLong_Check(a[6])) Py_RETURN_NONE;
  const Tensor *table = tensor(a[0]), *held = tensor(a[1]), *wanted = tensor(a[2]), *pages = tensor(a[3]),
               *free = tensor(a[4]);
  if (table == nullptr || table->dim() != 2 || pages == nullptr || pages->dim() != 1) Py_RETURN_NONE;
  const int64_t B = table->size(0), blocks = table->size(1), P = pages->size(0);
  int overflow = 0;
  const long long page = PyLong_AsLongLongAndOverflow(a[5], &overflow);
  if (overflow != 0 || page < INT32_MIN || page > INT32_MAX) Py_RETURN_NONE;
  const long long T = PyLong_AsLongLongAndOverflow(a[6], &overflow);
  if (overflow != 0 || T < 0 || T > INT32_MAX || B >= INT32_MAX || blocks > INT32_MAX || P > INT32_MAX ||
      !dense(table, at::kInt, {B, blocks}) || !ints(held, B) || !ints(wanted, B) || !ints(pages, P) || !ints(free, 1))
    Py_RETURN_NONE;
  const int64_t sizes[4] = {B, B + 1, T, T};
  Tensor out[4];
  bool fresh = true;
  for (int i = 0; i < 4; ++i) fresh = fresh && a[7 + i] == Py_None;
  int64_t total = 0, at[4];
  for (int i = 0; i < 4; ++i) at[i] = total, total += (sizes[i] + 63) / 64 * 64;
  if (fresh && total * 4 <= kShared && T > 0) {  // one allocation
    Tensor all = empty({total}, at::kInt, *table);
    for (int i = 0; i < 4; ++i) {
      out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                        c10::scalarTypeToTypeMeta(at::kInt));
      out[i].unsafeGetTensorImpl()->set_storage_offset(at[i]);
      out[i].unsafeGetTensorImpl()->set_sizes_contiguous({sizes[i]});
    }
  } else {
    for (int i = 0; i < 4; ++i)
      if (!output(a[7 + i], {sizes[i]}, at::kInt, *table, &out[i])) Py_RETURN_NONE;
  }
  int* p[4];
  for (int i = 0; i < 4; ++i) p[i] = (int*)out[i].data_ptr();
  const attn_status s = attn_cache_reserve((int*)table->data_ptr(), (const int*)held->data_ptr(),
                                           (const int*)wanted->data_ptr(), (int*)pages->data_ptr(),
                                           (int*)free->data_ptr(), p[0], p[1], p[2], p[3], (int)B, (int)T, (int)P,
                                           (int)page, (int)blocks, stream());
  if (s != ATTN_OK) return raise("attn_cache_reserve", s);
  PyObject* r = PyTuple_New(4);
  for (int i = 0; r != nullptr && i < 4; ++i) {
    PyObject* x = THPVariable_Wrap(out[i]);
    if (x == nullptr) Py_CLEAR(r);
    else PyTuple_SET_ITEM(r, i, x);
  }
  return r;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"varlen_fwd", (PyCFunction)(void (*)())varlen_fwd, METH_FASTCALL, nullptr},
    {"cache_append", (PyCFunction)(void (*)())cache_append, METH_FASTCALL, nullptr},
    {"cache_read", (PyCFunction)(void (*)())cache_read, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)())decode, METH_FASTCALL, nullptr},
    {"decode_shared", (PyCFunction)(void (*)())decode_shared, METH_FASTCALL, nullptr},
    {"cache_reserve", (PyCFunction)(void (*)())cache_reserve, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__attn_torch(void) { return PyModule_Create(&module); }
