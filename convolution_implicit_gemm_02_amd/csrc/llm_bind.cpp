// llm_bind.cpp -- the Python extension module _llm_bind: calls of the decoder-step operators whose arguments are in order, with
// little cost to the host.  It looks at the same things as llm.py and never decides that something is wrong: it returns -1,
// and llm.py says what.  A call of one token costs the GPU 2 to 10 us; from Python statements alone the host needs 8, so 5.
#include <Python.h>
#include <algorithm>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cbs_llm.h"

namespace {

using Sizes = std::initializer_list<int64_t>;

decltype(&cbs_rms_norm) fn_rms_norm;
decltype(&cbs_w4_linear) fn_w4_linear;
decltype(&cbs_kv_write) fn_kv_write;
decltype(&cbs_kv_read) fn_kv_read;
decltype(&cbs_attn_run) fn_attn_run;

at::ScalarType kind_of(int t) {
  switch (t) {
    case CBS_F32: return at::kFloat;
    case CBS_I8: return at::kChar;
    case CBS_F16: return at::kHalf;
    case CBS_BF16: return at::kBFloat16;
    default: return at::ScalarType::Undefined;
  }
}

// The arguments of one call: what is looked up is remembered as wrong once it is.
struct Call {
  PyObject *const *args;
  bool ok = true;
  int dev = -1;

  const at::Tensor *tensor(int i) {
    if (!THPVariable_Check(args[i])) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(args[i]);
  }
  // its device is the call's: the current one
  bool first(const at::Tensor *t) {
    if (!t || !t->is_cuda() || t->get_device() != c10::hip::current_device()) return ok = false;
    dev = (int)t->get_device();
    return true;
  }
  // dense throughout, or in its last axis; a missing tensor that may be missing is null
  void *at(int i, at::ScalarType kind, Sizes sizes, bool dense, bool may_miss = false) {
    if (may_miss && args[i] == Py_None) return nullptr;
    const at::Tensor *t = tensor(i);
    if (!t) return nullptr;
    if (t->scalar_type() != kind || t->sizes() != c10::IntArrayRef(sizes) || !t->is_cuda() || t->get_device() != dev ||
        !(t->is_contiguous() || (!dense && (t->stride(-1) == 1 || t->size(-1) <= 1)))) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  int64_t stride(int i, int axis) { return args[i] == Py_None ? 0 : THPVariable_Unpack(args[i]).stride(axis); }
  void *stream() { return (void *)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }
};

// A descriptor is a ctypes structure.
template <typename D>
bool read_desc(PyObject *o, D *d) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return false;
  }
  const bool fits = b.len == (Py_ssize_t)sizeof(D);
  if (fits) memcpy(d, b.buf, sizeof(D));
  PyBuffer_Release(&b);
  return fits;
}

PyObject *answer(long v) { return PyLong_FromLong(v); }

// desc, x, weight, out, residual, residual_out, out_scale
PyObject *rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
  cbs_rms_desc d;
  Call c{args};
  const at::Tensor *x = n == 7 && read_desc(args[0], &d) ? c.tensor(1) : nullptr;
  if (!c.first(x) || x->dim() != 2 || x->size(1) != d.dim) return answer(-1);
  const int64_t rows = x->size(0);
  const at::ScalarType kind = kind_of(d.dtype);
  cbs_rms_args a;
  a.x = c.at(1, kind, {rows, d.dim}, false);
  a.weight = c.at(2, kind_of(d.weight_dtype), {d.dim}, true);
  a.out = c.at(3, kind_of(d.out_dtype), {rows, d.dim}, false);
  a.residual = c.at(4, kind, {rows, d.dim}, false, true);
  a.residual_out = c.at(5, kind, {rows, d.dim}, false, true);
  a.out_scale = (float *)c.at(6, at::kFloat, {rows}, true, true);
  if (!c.ok) return answer(-1);
  a.rows = rows;
  a.x_stride = c.stride(1, 0), a.residual_stride = c.stride(4, 0), a.out_stride = c.stride(3, 0), a.residual_out_stride = c.stride(5, 0);
  return answer(fn_rms_norm(&d, &a, c.stream()));
}

// desc, x, codes, scales, out, zeros, x_scale
PyObject *w4_linear(PyObject *, PyObject *const *args, Py_ssize_t n) {
  cbs_w4_desc d;
  Call c{args};
  const at::Tensor *x = n == 7 && read_desc(args[0], &d) ? c.tensor(1) : nullptr;
  if (!c.first(x) || x->dim() != 2 || d.group < 1 || d.k < 1) return answer(-1);
  const int64_t rows = x->size(0), groups = ((int64_t)d.k + d.group - 1) / d.group;
  cbs_w4_args a;
  a.x = c.at(1, kind_of(d.dtype), {rows, d.k}, false);
  a.codes = (const uint8_t *)c.at(2, at::kByte, {d.n, ((int64_t)d.k + 31) / 32 * 16}, true);
  a.scales = c.at(3, kind_of(d.scale_dtype), {groups, d.n}, true);
  a.out = c.at(4, kind_of(d.out_dtype), {rows, d.n}, false);
  a.zeros = (const uint8_t *)c.at(5, at::kByte, {groups, d.n}, true, true);
  a.x_scale = (const float *)c.at(6, at::kFloat, {rows}, true, true);
  if (!c.ok) return answer(-1);
  a.rows = rows;
  a.x_stride = c.stride(1, 0), a.out_stride = c.stride(4, 0);
  return answer(fn_w4_linear(&d, &a, c.stream()));
}

// desc, k, v, slots, k_cache, v_cache, k_scale, v_scale
PyObject *kv(PyObject *const *args, Py_ssize_t n, bool write) {
  cbs_kv_desc d;
  Call c{args};
  const at::Tensor *slots = n == 8 && read_desc(args[0], &d) ? c.tensor(3) : nullptr;
  if (!c.first(slots) || slots->dim() != 1) return answer(-1);
  const at::Tensor *cache = c.tensor(4);
  if (!cache || cache->dim() != 4) return answer(-1);
  const int64_t tokens = slots->size(0), pages = cache->size(0);
  const at::ScalarType kind = kind_of(write ? d.dtype : d.read_dtype), kept = kind_of(d.cache_dtype);
  cbs_kv_args a;
  a.k = c.at(1, kind, {tokens, d.heads, d.head_dim}, false);
  a.v = c.at(2, kind, {tokens, d.heads, d.head_dim}, false);
  a.slots = (const int64_t *)c.at(3, at::kLong, {tokens}, true);
  a.k_cache = c.at(4, kept, {pages, d.heads, d.page_size, d.head_dim}, true);
  a.v_cache = c.at(5, kept, {pages, d.heads, d.head_dim, d.page_size}, true);
  a.k_scale = (float *)c.at(6, at::kFloat, {pages, d.heads, d.page_size}, true, true);
  a.v_scale = (float *)c.at(7, at::kFloat, {pages, d.heads, d.page_size}, true, true);
  if (!c.ok) return answer(-1);
  a.tokens = tokens, a.pages = pages;
  a.k_token_stride = c.stride(1, 0), a.k_head_stride = c.stride(1, 1), a.v_token_stride = c.stride(2, 0), a.v_head_stride = c.stride(2, 1);
  return answer((write ? fn_kv_write : fn_kv_read)(&d, &a, c.stream()));
}
PyObject *kv_write(PyObject *, PyObject *const *args, Py_ssize_t n) { return kv(args, n, true); }
PyObject *kv_read(PyObject *, PyObject *const *args, Py_ssize_t n) { return kv(args, n, false); }

// handle, desc, q, q_start, kv_len, table, k_cache, v_cache, out, k_scale, v_scale, max_new, max_kv
PyObject *attn_run(PyObject *, PyObject *const *args, Py_ssize_t n) {
  cbs_attn_desc d;
  Call c{args};
  const at::Tensor *q = n == 13 && read_desc(args[1], &d) ? c.tensor(2) : nullptr;
  if (!c.first(q) || q->dim() != 3) return answer(-1);
  const at::Tensor *table = c.tensor(5), *cache = c.tensor(6);
  if (!table || table->dim() != 2 || !cache || cache->dim() != 4) return answer(-1);
  const int64_t tokens = q->size(0), seqs = table->size(0), columns = table->size(1), pages = cache->size(0);
  const at::ScalarType kind = kind_of(d.dtype), kept = kind_of(d.cache_dtype);
  cbs_attn_args a;
  a.q = c.at(2, kind, {tokens, d.heads, d.head_dim}, false);
  a.q_start = (const int32_t *)c.at(3, at::kInt, {seqs + 1}, true);
  a.kv_len = (const int32_t *)c.at(4, at::kInt, {seqs}, true);
  a.table = (const int32_t *)c.at(5, at::kInt, {seqs, columns}, false);
  a.k_cache = c.at(6, kept, {pages, d.kv_heads, d.page_size, d.head_dim}, true);
  a.v_cache = c.at(7, kept, {pages, d.kv_heads, d.head_dim, d.page_size}, true);
  a.out = c.at(8, kind, {tokens, d.heads, d.head_dim}, false);
  a.k_scale = (const float *)c.at(9, at::kFloat, {pages, d.kv_heads, d.page_size}, true, true);
  a.v_scale = (const float *)c.at(10, at::kFloat, {pages, d.kv_heads, d.page_size}, true, true);
  void *handle = PyLong_Check(args[0]) ? PyLong_AsVoidPtr(args[0]) : nullptr;
  long most[2];
  const int64_t all[2] = {tokens == seqs ? 1 : tokens, std::min<int64_t>(columns * d.page_size, 0x7fffffff)};
  for (int i = 0; i < 2; i++) {
    int over = 0;
    most[i] = args[11 + i] == Py_None ? (long)all[i] : PyLong_Check(args[11 + i]) ? PyLong_AsLongAndOverflow(args[11 + i], &over) : -1;
    if (over || most[i] < 0 || most[i] > 0x7fffffff) c.ok = false;
  }
  if (PyErr_Occurred()) PyErr_Clear(), c.ok = false;
  if (!c.ok || !handle || seqs > 0x7fffffff || columns > 0x7fffffff) return answer(-1);
  a.tokens = tokens, a.pages = pages;
  a.q_token_stride = c.stride(2, 0), a.q_head_stride = c.stride(2, 1), a.out_token_stride = c.stride(8, 0), a.out_head_stride = c.stride(8, 1);
  a.table_stride = c.stride(5, 0);
  a.seqs = (int32_t)seqs, a.columns = (int32_t)columns, a.max_new = (int32_t)most[0], a.max_kv = (int32_t)most[1];
  return answer(fn_attn_run((const cbs_attn *)handle, &a, c.stream()));
}

// Addresses of the library's entry points, which llm.py has loaded.
PyObject *setup(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *at[5] = {};
  for (Py_ssize_t i = 0; i < 5 && i < n; i++) at[i] = PyLong_AsVoidPtr(args[i]);
  if (PyErr_Occurred()) return nullptr;
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "five addresses");
    return nullptr;
  }
  fn_rms_norm = (decltype(fn_rms_norm))at[0];
  fn_w4_linear = (decltype(fn_w4_linear))at[1];
  fn_kv_write = (decltype(fn_kv_write))at[2];
  fn_kv_read = (decltype(fn_kv_read))at[3];
  fn_attn_run = (decltype(fn_attn_run))at[4];
  Py_RETURN_NONE;
}

// No C++ exception leaves an entry: what torch throws is the slower way's to report.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (...) {
    return answer(-1);
  }
}

#define ENTRY(f) {#f, (PyCFunction)(void (*)(void))guarded<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(setup), ENTRY(rms_norm), ENTRY(w4_linear), ENTRY(kv_write), ENTRY(kv_read), ENTRY(attn_run), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_llm_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__llm_bind(void) { return PyModule_Create(&module); }
