// Reads tensors for the wrappers of the serving operators: type, device, sizes and strides checked
// and turned into the C ABI's structs, in one call each.
//
// A small operator's call is bound by the host.  Asked from Python, one tensor's type, device,
// sizes, strides and address take 0.5 us, here 0.1, and a call names ten tensors: an append of
// 16 tokens (4.2 us of kernel) takes 7.3 us instead of 11.5, a gated delta step of one (4.4) 7.2
// instead of 9.3.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <string>

#include "../include/attn.h"
#include "../include/pages.h"

namespace {

struct Refused {
  std::string why;
};
[[noreturn]] void refuse(const std::string &why) { throw Refused{why}; }

const at::Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": a tensor required");
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject *o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}
std::string sizes_text(const int64_t *n, int dims) {
  std::string s;
  for (int i = 0; i < dims; ++i) s += n[i] < 0 ? "[]" : "[" + std::to_string(n[i]) + "]";
  return s;
}
std::string type_text(int64_t type) { return c10::toString((at::ScalarType)type); }

// A negative size: any; no sizes at all: of any shape.
bool sizes_are(const at::Tensor &t, const int64_t *n, int dims) {
  if (dims > 0 && t.dim() != dims) return false;
  for (int i = 0; i < dims; ++i)
    if (n[i] >= 0 && t.size(i) != n[i]) return false;
  return true;
}
int32_t small(const char *name, int64_t n) {
  if (n > INT32_MAX) refuse(std::string(name) + ": too large");
  return (int32_t)n;
}
// strides of dimensions of one element say nothing
int64_t stride(const at::Tensor &t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// Address of a contiguous tensor.
const void *address(const char *name, PyObject *o, at::ScalarType type, int64_t index, const int64_t *n, int dims) {
  const at::Tensor &t = tensor(name, o);
  if (t.scalar_type() != type || index < 0 || t.get_device() != index || !sizes_are(t, n, dims) || !t.is_contiguous())
    refuse(std::string(name) + ": contiguous " + type_text((int64_t)type) + " " + sizes_text(n, dims) + " on cuda:" +
           std::to_string(index) + " required");
  return t.data_ptr();
}

// f(name, ...) with its exceptions turned into Python's.
template <class F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t least, F f) {
  HANDLE_TH_ERRORS
  try {
    if (given < least) refuse("too few arguments");
    return f();
  } catch (const Refused &r) {
    PyErr_SetString(PyExc_ValueError, r.why.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
const char *text(PyObject *o) {
  const char *s = PyUnicode_AsUTF8(o);
  if (!s) throw python_error();
  return s;
}
template <class T>
PyObject *bytes(const T &x) {
  return PyBytes_FromStringAndSize((const char *)&x, sizeof x);
}

// address(name, tensor, type, index, sizes...): address of a contiguous tensor; a size of -1: any, no
// sizes: any shape
PyObject *py_address(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    int64_t sizes[8];
    const int dims = (int)(n - 4);
    if (dims > 8) refuse("too many sizes");
    for (int i = 0; i < dims; ++i) sizes[i] = integer(a[4 + i]);
    return PyLong_FromVoidPtr(
        const_cast<void *>(address(text(a[0]), a[1], (at::ScalarType)integer(a[2]), integer(a[3]), sizes, dims)));
  });
}

// heads(name, tensor, T, heads, D, type, index): (moe_heads, T, heads); T or heads -1: any
PyObject *py_heads(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const char *name = text(a[0]);
    const at::Tensor &t = tensor(name, a[1]);
    const int64_t sizes[3] = {integer(a[2]), integer(a[3]), integer(a[4])}, type = integer(a[5]), index = integer(a[6]);
    if ((int64_t)t.scalar_type() != type || index < 0 || t.get_device() != index || !sizes_are(t, sizes, 3))
      refuse(std::string(name) + ": " + type_text(type) + " " + sizes_text(sizes, 3) + " on cuda:" + std::to_string(index) +
             " required");
    if (t.stride(2) != 1) refuse(std::string(name) + ": contiguous last dimension required");
    const moe_heads h{t.data_ptr(), stride(t, 0), stride(t, 1)};
    return Py_BuildValue("NLi", bytes(h), (long long)t.size(0), small(name, t.size(1)));
  });
}

// cache(k, v, index): (moe_paged_kv, KV heads, head width, type)
PyObject *py_cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    const at::Tensor &k = tensor("k_cache", a[0]), &v = tensor("v_cache", a[1]);
    const int64_t index = integer(a[2]);
    const at::ScalarType type = k.scalar_type();
    if ((type != at::kBFloat16 && type != at::kHalf) || index < 0 || k.get_device() != index || k.dim() != 4)
      refuse("k_cache: bfloat16 or float16 [n_pages][page_size][n_kv_heads][head_dim] on q's GPU required");
    if (v.scalar_type() != type || v.get_device() != index || v.sizes() != k.sizes())
      refuse("v_cache must have k_cache's type, device and shape");
    if (v.strides() != k.strides() || k.stride(3) != 1)
      refuse("k_cache and v_cache must have the same strides and a contiguous last dimension");
    moe_paged_kv kv{};
    kv.k = k.data_ptr();
    kv.v = v.data_ptr();
    kv.page_stride = stride(k, 0);
    kv.token_stride = stride(k, 1);
    kv.head_stride = stride(k, 2);
    kv.n_pages = small("k_cache", k.size(0));
    kv.page_size = small("k_cache", k.size(1));
    kv.n_kv_heads = small("k_cache", k.size(2));
    kv.head_dim = small("k_cache", k.size(3));
    kv.dtype = type == at::kHalf ? MOE_FP16 : MOE_BF16;
    return Py_BuildValue("Niii", bytes(kv), kv.n_kv_heads, kv.head_dim, (int)type);
  });
}

// batch(table, q_start, kv_len, row or None, index): (moe_batch, sequences)
PyObject *py_batch(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    const int64_t index = integer(a[4]), any[2] = {-1, -1};
    moe_batch b{};
    b.table = (const int32_t *)address("table", a[0], at::kInt, index, any, 2);
    b.q_start = (const int32_t *)address("q_start", a[1], at::kInt, index, any, 1);
    const at::Tensor &table = THPVariable_Unpack(a[0]);
    const int64_t rows = table.size(0), seqs = THPVariable_Unpack(a[1]).size(0) - 1;
    b.kv_len = (const int32_t *)address("kv_len", a[2], at::kInt, index, &rows, 1);
    if (a[3] != Py_None) b.row = (const int32_t *)address("row", a[3], at::kInt, index, &seqs, 1);
    b.n_seqs = small("q_start", seqs);
    b.n_rows = small("table", rows);
    b.table_cols = small("table", table.size(1));
    return Py_BuildValue("Ni", bytes(b), b.n_seqs);
  });
}

// memory(cache, n_pages, index): moe_page_memory of a cache [n_planes][n_pages][...]
PyObject *py_memory(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    const at::Tensor &c = tensor("cache", a[0]);
    const int64_t pages = integer(a[1]), index = integer(a[2]);
    if (index < 0 || c.get_device() != index || c.dim() < 3 || c.size(1) != pages || c.size(0) < 1)
      refuse("cache: [n_planes][" + std::to_string(pages) + "][...] on the pool's GPU required");
    int64_t page = 1;
    for (int64_t d = c.dim() - 1; d >= 2; --d) {
      if (c.size(d) != 1 && c.stride(d) != page) refuse("cache: each page must be contiguous");
      page *= c.size(d);
    }
    const int64_t size = c.element_size();
    moe_page_memory m{};
    m.base = c.data_ptr();
    m.plane_stride = stride(c, 0) * size;
    m.page_stride = stride(c, 1) * size;
    m.page_bytes = page * size;
    m.n_planes = small("cache", c.size(0));
    return bytes(m);
  });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyCFunction fast() {
  return (PyCFunction)(void (*)(void))F;
}
PyMethodDef methods[] = {{"address", fast<py_address>(), METH_FASTCALL, nullptr},
                         {"heads", fast<py_heads>(), METH_FASTCALL, nullptr},
                         {"cache", fast<py_cache>(), METH_FASTCALL, nullptr},
                         {"batch", fast<py_batch>(), METH_FASTCALL, nullptr},
                         {"memory", fast<py_memory>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
  PyObject *m = PyModule_Create(&module);
  const struct {
    const char *name;
    at::ScalarType type;
  } types[] = {{"BF16", at::kBFloat16}, {"FP16", at::kHalf}, {"FP32", at::kFloat},
               {"FP64", at::kDouble},   {"INT32", at::kInt}, {"UINT8", at::kByte}};
  for (const auto &t : types)
    if (m) PyModule_AddIntConstant(m, t.name, (long)t.type);
  return m;
}
