// bind.cpp -- the Python side of the cache operators: checks torch tensors and
// calls the C ABI with their addresses and strides.
//
// A cache operator's kernel takes a few microseconds for one sequence, and reading
// its tensors' attributes from Python took about as long again (a commit call: 7.0
// us through ctypes, 2.8 here).  Nothing but argument marshalling happens here.  The
// entry points' addresses come from the loaded libdflash2.so (init), so that this
// module needs no link to it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "dflash2.h"

namespace {

decltype(&dflash2_tree_attention) f_attention = nullptr;
decltype(&dflash2_cache_commit) f_commit = nullptr;
decltype(&dflash2_cache_scores) f_scores = nullptr;
decltype(&dflash2_cache_evict) f_evict = nullptr;

// A failed check: the Python error has been set.
struct Refused {};

[[noreturn]] void refuse(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s: %s", name, what);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
  return t;
}

bool is_bf16(const at::Tensor& t) {
  const auto s = t.scalar_type();
  return s == at::kBFloat16 || s == at::kShort || s == at::kUInt16;
}

uint16_t* bits(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }

// A contiguous tensor of one type and shape.
void* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type) refuse(name, "wrong type");
  if (t.sizes() != shape) refuse(name, "wrong shape");
  if (!t.is_contiguous()) refuse(name, "expected a contiguous tensor");
  return t.data_ptr();
}
void* dense_or_null(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  return o == Py_None ? nullptr : dense(o, name, type, shape);
}

// A bf16 [B, T, heads, dim] operand with unit stride along its last dimension.
const at::Tensor& rows(PyObject* o, const char* name, int64_t dim) {
  const at::Tensor& t = tensor(o, name);
  if (!is_bf16(t) || t.dim() != 4 || t.size(3) != dim || t.stride(3) != 1)
    refuse(name, "expected bf16 [B, T, heads, dim] of the cache's dim, unit stride along the last dimension");
  return t;
}

// The drafted nodes' keys and values: one shape, one layout.
void pair(const at::Tensor& k, const at::Tensor& v, int64_t B, int64_t T, int64_t heads) {
  if (k.size(0) != B || k.size(1) != T || k.size(2) != heads || v.sizes() != k.sizes() || v.strides() != k.strides())
    refuse("k_new, v_new", "expected [B, T, kv_heads, dim] with equal strides");
}

template <class T>
T* address(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refused();
  return reinterpret_cast<T*>(static_cast<intptr_t>(x));
}
int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refused();
  return x;
}
float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(x);
}

void sequences(int64_t have, int64_t want, const char* name) {
  if (have < want) refuse(name, "fewer sequences than the call's");
}

// Runs a call's body; no C++ exception reaches Python.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, const F& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// handle, cache, cache_batch, q, cache_len, k_new, v_new, tree_mask, scale, out, lse, workspace, stream
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() {
    const auto* cache = address<dflash2_kv_cache>(a[1]);
    const at::Tensor& q = rows(a[3], "q", cache->head_dim);
    const int64_t B = q.size(0), T = q.size(1), heads = q.size(2);
    sequences(integer(a[2]), B, "cache");
    const uint16_t *k = nullptr, *v = nullptr;
    int64_t ns[3] = {0, 0, 0};
    if ((a[5] == Py_None) != (a[6] == Py_None)) refuse("k_new, v_new", "both or neither");
    if (a[5] != Py_None) {
      const at::Tensor &kn = rows(a[5], "k_new", cache->head_dim), &vn = rows(a[6], "v_new", cache->head_dim);
      pair(kn, vn, B, T, cache->heads);
      k = bits(kn);
      v = bits(vn);
      for (int i = 0; i < 3; ++i) ns[i] = kn.stride(i);
    }
    const at::Tensor& out = tensor(a[9], "out");
    if (!is_bf16(out) || out.sizes() != q.sizes() || !out.is_contiguous()) refuse("out", "expected contiguous bf16 of q's shape");
    const at::Tensor& ws = tensor(a[11], "workspace");
    if (!ws.is_contiguous()) refuse("workspace", "expected a contiguous tensor");
    return f_attention(address<dflash2_handle>(a[0]), bits(q), q.stride(0), q.stride(1), q.stride(2), cache,
                       static_cast<int32_t*>(dense(a[4], "cache_len", at::kInt, {B})), k, v, ns[0], ns[1], ns[2],
                       static_cast<uint64_t*>(dense_or_null(a[7], "tree_mask", at::kLong, {B, T, (T + 63) / 64})), B, T,
                       heads, number(a[8]), bits(out),
                       static_cast<float*>(dense(a[10], "lse", at::kFloat, {B, T, heads})), ws.data_ptr(), ws.nbytes(),
                       address<void>(a[12]));
  });
}

// handle, cache, cache_batch, k_new, v_new, cache_len, count, path, scores, new_len, stream
PyObject* cache_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() {
    const auto* cache = address<dflash2_kv_cache>(a[1]);
    const at::Tensor &k = rows(a[3], "k_new", cache->head_dim), &v = rows(a[4], "v_new", cache->head_dim);
    const int64_t B = k.size(0), T = k.size(1);
    pair(k, v, B, T, cache->heads);
    sequences(integer(a[2]), B, "cache");
    float* scores = nullptr;
    int64_t ld = 0;
    if (a[8] != Py_None) {
      const at::Tensor& s = tensor(a[8], "scores");
      ld = s.dim() == 3 ? s.size(2) : 0;
      scores = static_cast<float*>(dense(a[8], "scores", at::kFloat, {B, cache->heads, ld}));
    }
    return f_commit(address<dflash2_handle>(a[0]), bits(k), bits(v), k.stride(0), k.stride(1), k.stride(2), cache,
                    static_cast<int32_t*>(dense(a[5], "cache_len", at::kInt, {B})),
                    static_cast<int32_t*>(dense_or_null(a[6], "count", at::kInt, {B})),
                    static_cast<int32_t*>(dense_or_null(a[7], "path", at::kInt, {B, T})), B, T, scores, ld,
                    static_cast<int32_t*>(dense(a[9], "new_len", at::kInt, {B})), address<void>(a[10]));
  });
}

// handle, cache, cache_batch, q, lse, cache_len, scores, count, path, scale, stream
PyObject* cache_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() {
    const auto* cache = address<dflash2_kv_cache>(a[1]);
    const at::Tensor& q = rows(a[3], "q", cache->head_dim);
    const int64_t B = q.size(0), T = q.size(1), heads = q.size(2);
    sequences(integer(a[2]), B, "cache");
    const at::Tensor& s = tensor(a[6], "scores");
    const int64_t ld = s.dim() == 3 ? s.size(2) : 0;
    return f_scores(address<dflash2_handle>(a[0]), bits(q), q.stride(0), q.stride(1), q.stride(2),
                    static_cast<float*>(dense(a[4], "lse", at::kFloat, {B, T, heads})), cache,
                    static_cast<int32_t*>(dense(a[5], "cache_len", at::kInt, {B})),
                    static_cast<int32_t*>(dense_or_null(a[7], "count", at::kInt, {B})),
                    static_cast<int32_t*>(dense_or_null(a[8], "path", at::kInt, {B, T})), B, T, heads, number(a[9]),
                    static_cast<float*>(dense(a[6], "scores", at::kFloat, {B, cache->heads, ld})), ld,
                    address<void>(a[10]));
  });
}

// handle, cache, cache_batch, dst, dst_batch, scores, cache_len, keep, recent, kept, new_len, dst_scores, stream
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() {
    const auto *cache = address<dflash2_kv_cache>(a[1]), *dst = address<dflash2_kv_cache>(a[3]);
    const at::Tensor& s = tensor(a[5], "scores");
    const int64_t B = s.dim() == 3 ? s.size(0) : 0, ld = s.dim() == 3 ? s.size(2) : 0, heads = cache->heads;
    sequences(integer(a[2]), B, "cache");
    sequences(integer(a[4]), B, "dst");
    const int64_t keep = integer(a[7]);
    float* dst_scores = nullptr;
    int64_t dst_ld = keep;
    if (a[11] != Py_None) {
      const at::Tensor& d = tensor(a[11], "dst_scores");
      dst_ld = d.dim() == 3 ? d.size(2) : 0;
      dst_scores = static_cast<float*>(dense(a[11], "dst_scores", at::kFloat, {B, heads, dst_ld}));
    }
    return f_evict(address<dflash2_handle>(a[0]),
                   static_cast<float*>(dense(a[5], "scores", at::kFloat, {B, heads, ld})), ld, cache,
                   static_cast<int32_t*>(dense(a[6], "cache_len", at::kInt, {B})), dst, B, keep, integer(a[8]),
                   static_cast<int32_t*>(dense(a[9], "kept", at::kInt, {B, heads, keep > 0 ? keep : 0})),
                   static_cast<int32_t*>(dense(a[10], "new_len", at::kInt, {B})), dst_scores, dst_ld,
                   address<void>(a[12]));
  });
}

// addresses of the four entry points, in this order
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() {
    f_attention = reinterpret_cast<decltype(f_attention)>(integer(a[0]));
    f_commit = reinterpret_cast<decltype(f_commit)>(integer(a[1]));
    f_scores = reinterpret_cast<decltype(f_scores)>(integer(a[2]));
    f_evict = reinterpret_cast<decltype(f_evict)>(integer(a[3]));
    return 0;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<init>("init"),
                         method<tree_attention>("tree_attention"),
                         method<cache_commit>("cache_commit"),
                         method<cache_scores>("cache_scores"),
                         method<cache_evict>("cache_evict"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dflash2_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dflash2_bind() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose tensors it reads: another one's may be laid out otherwise
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", DFLASH2_TORCH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
