// bind.cpp -- the Python side of the cache operators and of those around them (rotary
// positions, appending, logits, counts): checks torch tensors and calls the C ABI with their
// addresses and strides.
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
decltype(&dflash2_prefix_attention) f_prefix = nullptr;
decltype(&dflash2_rope) f_rope = nullptr;
decltype(&dflash2_cache_append) f_append = nullptr;
decltype(&dflash2_logits_adjust) f_logits = nullptr;
decltype(&dflash2_token_counts) f_counts = nullptr;

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

// A call's tensors have to be on the handle's device.
const at::Tensor& here(const at::Tensor& t, int64_t device, const char* name) {
  if (t.get_device() != device) refuse(name, "expected a tensor on the handle's device");
  return t;
}
const at::Tensor& here(PyObject* o, int64_t device, const char* name) { return here(tensor(o, name), device, name); }
template <class T>
T* dense_here(PyObject* o, int64_t device, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  if (o == Py_None) return nullptr;
  here(o, device, name);
  return static_cast<T*>(dense(o, name, type, shape));
}

// A bf16 [B, T, heads, dim] tensor with unit stride along its last dimension.
const at::Tensor& heads_of(PyObject* o, int64_t device, const char* name) {
  const at::Tensor& t = here(o, device, name);
  if (!is_bf16(t) || t.dim() != 4 || (t.stride(3) != 1 && t.size(3) != 1))
    refuse(name, "expected bf16 [B, T, heads, dim], unit stride along the last dimension");
  return t;
}

// A two- or three-dimensional operand with columns at unit stride.
const at::Tensor& columns(PyObject* o, int64_t device, const char* name, int64_t dims) {
  const at::Tensor& t = here(o, device, name);
  if (t.dim() != dims || (t.stride(dims - 1) != 1 && t.size(dims - 1) != 1)) refuse(name, "wrong shape or strides");
  return t;
}

// handle, device, rope, x, out, base, depth, inverse, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() {
    const int64_t device = integer(a[1]);
    const at::Tensor &x = heads_of(a[3], device, "x"), &out = heads_of(a[4], device, "out");
    if (out.sizes() != x.sizes()) refuse("out", "expected x's shape");
    const int64_t B = x.size(0), T = x.size(1);
    return f_rope(address<dflash2_handle>(a[0]), address<dflash2_rope_table>(a[2]), bits(x), x.stride(0), x.stride(1),
                  x.stride(2), bits(out), out.stride(0), out.stride(1), out.stride(2),
                  dense_here<int32_t>(a[5], device, "base", at::kInt, {B}),
                  dense_here<int32_t>(a[6], device, "depth", at::kInt, {B, T}), B, T, x.size(2), x.size(3),
                  static_cast<int>(integer(a[7])), address<void>(a[8]));
  });
}

// handle, device, cache, cache_batch, k_new, v_new, cache_len, rope, count, position, q, q_out, scores, new_len, stream
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() {
    const int64_t device = integer(a[1]);
    const auto* cache = address<dflash2_kv_cache>(a[2]);
    const at::Tensor &k = here(rows(a[4], "k_new", cache->head_dim), device, "k_new"),
                     &v = here(rows(a[5], "v_new", cache->head_dim), device, "v_new");
    const int64_t B = k.size(0), T = k.size(1);
    pair(k, v, B, T, cache->heads);
    sequences(integer(a[3]), B, "cache");
    const uint16_t* q = nullptr;
    uint16_t* q_out = nullptr;
    int64_t qs[3] = {0, 0, 0}, os[3] = {0, 0, 0}, heads = 0;
    if ((a[10] == Py_None) != (a[11] == Py_None)) refuse("q, q_out", "both or neither");
    if (a[10] != Py_None) {
      const at::Tensor &x = heads_of(a[10], device, "q"), &y = heads_of(a[11], device, "q_out");
      heads = x.size(2);
      if (x.sizes() != y.sizes() || x.size(0) != B || x.size(1) != T || x.size(3) != cache->head_dim)
        refuse("q, q_out", "expected [B, T, heads, dim] of k_new's B, T and dim");
      q = bits(x);
      q_out = bits(y);
      for (int i = 0; i < 3; ++i) qs[i] = x.stride(i), os[i] = y.stride(i);
    }
    float* scores = nullptr;
    int64_t ld = 0;
    if (a[12] != Py_None) {
      const at::Tensor& s = here(a[12], device, "scores");
      ld = s.dim() == 3 ? s.size(2) : 0;
      scores = static_cast<float*>(dense(a[12], "scores", at::kFloat, {B, cache->heads, ld}));
    }
    if (a[6] == Py_None || a[13] == Py_None) refuse("cache_len, new_len", "expected a tensor");
    return f_append(address<dflash2_handle>(a[0]), bits(k), bits(v), k.stride(0), k.stride(1), k.stride(2), cache,
                    dense_here<int32_t>(a[6], device, "cache_len", at::kInt, {B}), address<dflash2_rope_table>(a[7]),
                    dense_here<int32_t>(a[8], device, "count", at::kInt, {B}),
                    dense_here<int32_t>(a[9], device, "position", at::kInt, {B}), B, T, q, qs[0], qs[1], qs[2], q_out,
                    os[0], os[1], os[2], heads, scores, ld,
                    dense_here<int32_t>(a[13], device, "new_len", at::kInt, {B}), address<void>(a[14]));
  });
}

// handle, device, logits, counts, tokens, tree_mask, repetition, frequency, presence, bias, allowed, out, stream
PyObject* logits_adjust(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() {
    const int64_t device = integer(a[1]);
    const at::Tensor &x = columns(a[2], device, "logits", 3), &out = columns(a[11], device, "out", 3);
    if (!is_bf16(x) || !is_bf16(out) || out.sizes() != x.sizes()) refuse("logits, out", "expected bf16 [B, T, V]");
    const int64_t B = x.size(0), T = x.size(1), V = x.size(2);
    const int32_t* counts = nullptr;
    const float* bias = nullptr;
    const uint32_t* allowed = nullptr;
    int64_t counts_ld = 0, bias_ld = 0, allowed_b = 0, allowed_t = 0;
    if (a[3] != Py_None) {
      const at::Tensor& t = columns(a[3], device, "counts", 2);
      if (t.scalar_type() != at::kInt || t.size(0) != B || t.size(1) != V) refuse("counts", "expected int32 [B, V]");
      counts = static_cast<int32_t*>(t.data_ptr());
      counts_ld = B > 1 ? t.stride(0) : V;
    }
    if (a[9] != Py_None) {
      const at::Tensor& t = columns(a[9], device, "bias", 2);
      if (t.scalar_type() != at::kFloat || (t.size(0) != B && t.size(0) != 1) || t.size(1) != V)
        refuse("bias", "expected fp32 [B, V] or [1, V]");
      bias = static_cast<float*>(t.data_ptr());
      bias_ld = t.size(0) > 1 ? t.stride(0) : 0;
    }
    if (a[10] != Py_None) {
      const at::Tensor& t = columns(a[10], device, "allowed", 3);
      if (t.scalar_type() != at::kInt || (t.size(0) != B && t.size(0) != 1) || (t.size(1) != T && t.size(1) != 1) ||
          t.size(2) != (V + 31) / 32)
        refuse("allowed", "expected int32 [B or 1, T or 1, (V + 31) // 32]");
      allowed = static_cast<uint32_t*>(t.data_ptr());
      allowed_b = t.size(0) > 1 ? t.stride(0) : 0;
      allowed_t = t.size(1) > 1 ? t.stride(1) : 0;
    }
    return f_logits(address<dflash2_handle>(a[0]), bits(x), x.stride(0), x.stride(1), B, T, V, counts, counts_ld,
                    dense_here<int32_t>(a[4], device, "tokens", at::kInt, {B, T}),
                    dense_here<uint64_t>(a[5], device, "tree_mask", at::kLong, {B, T, (T + 63) / 64}),
                    dense_here<float>(a[6], device, "repetition", at::kFloat, {B}),
                    dense_here<float>(a[7], device, "frequency", at::kFloat, {B}),
                    dense_here<float>(a[8], device, "presence", at::kFloat, {B}), bias, bias_ld, allowed, allowed_b,
                    allowed_t, bits(out), out.stride(0), out.stride(1), address<void>(a[12]));
  });
}

// handle, device, tokens, counts, count, path, prompt, stream
PyObject* token_counts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() {
    const int64_t device = integer(a[1]);
    const at::Tensor& tokens = here(a[2], device, "tokens");
    if (tokens.dim() != 2) refuse("tokens", "expected int32 [B, N]");
    const int64_t B = tokens.size(0), N = tokens.size(1);
    const at::Tensor& counts = columns(a[3], device, "counts", 2);
    if (counts.scalar_type() != at::kInt || counts.size(0) != B) refuse("counts", "expected int32 [B, V]");
    const int64_t V = counts.size(1);
    return f_counts(address<dflash2_handle>(a[0]), dense_here<int32_t>(a[2], device, "tokens", at::kInt, {B, N}),
                    dense_here<int32_t>(a[4], device, "count", at::kInt, {B}),
                    dense_here<int32_t>(a[5], device, "path", at::kInt, {B, N}), B, N, V, static_cast<int>(integer(a[6])),
                    static_cast<int32_t*>(counts.data_ptr()), B > 1 ? counts.stride(0) : V, address<void>(a[7]));
  });
}

// handle, device, cache, cache_batch, q, cache_len, prefix_len, prefix_start, k_new, v_new, tree_mask, scale, out, lse,
// workspace, stream
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() {
    const int64_t device = integer(a[1]);
    const auto* cache = address<dflash2_kv_cache>(a[2]);
    const at::Tensor& q = here(rows(a[4], "q", cache->head_dim), device, "q");
    const int64_t B = q.size(0), T = q.size(1), heads = q.size(2);
    sequences(integer(a[3]), B, "cache");
    const at::Tensor& shared = here(a[6], device, "prefix_len");
    if (shared.dim() != 1) refuse("prefix_len", "expected int32 [groups]");
    const int64_t groups = shared.size(0);
    const uint16_t *k = nullptr, *v = nullptr;
    int64_t ns[3] = {0, 0, 0};
    if ((a[8] == Py_None) != (a[9] == Py_None)) refuse("k_new, v_new", "both or neither");
    if (a[8] != Py_None) {
      const at::Tensor &kn = here(rows(a[8], "k_new", cache->head_dim), device, "k_new"),
                       &vn = here(rows(a[9], "v_new", cache->head_dim), device, "v_new");
      pair(kn, vn, B, T, cache->heads);
      k = bits(kn);
      v = bits(vn);
      for (int i = 0; i < 3; ++i) ns[i] = kn.stride(i);
    }
    const at::Tensor& out = here(a[12], device, "out");
    if (!is_bf16(out) || out.sizes() != q.sizes() || !out.is_contiguous()) refuse("out", "expected contiguous bf16 of q's shape");
    const at::Tensor& ws = here(a[14], device, "workspace");
    if (!ws.is_contiguous()) refuse("workspace", "expected a contiguous tensor");
    if (a[5] == Py_None) refuse("cache_len", "expected a tensor");
    return f_prefix(address<dflash2_handle>(a[0]), bits(q), q.stride(0), q.stride(1), q.stride(2), cache,
                    dense_here<int32_t>(a[5], device, "cache_len", at::kInt, {B}),
                    dense_here<int32_t>(a[6], device, "prefix_len", at::kInt, {groups}),
                    dense_here<int32_t>(a[7], device, "prefix_start", at::kInt, {groups + 1}), groups, k, v, ns[0], ns[1],
                    ns[2], dense_here<uint64_t>(a[10], device, "tree_mask", at::kLong, {B, T, (T + 63) / 64}), B, T, heads,
                    number(a[11]), bits(out), dense_here<float>(a[13], device, "lse", at::kFloat, {B, T, heads}),
                    ws.data_ptr(), ws.nbytes(), address<void>(a[15]));
  });
}

// addresses of the entry points, in this order
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() {
    f_attention = reinterpret_cast<decltype(f_attention)>(integer(a[0]));
    f_commit = reinterpret_cast<decltype(f_commit)>(integer(a[1]));
    f_scores = reinterpret_cast<decltype(f_scores)>(integer(a[2]));
    f_evict = reinterpret_cast<decltype(f_evict)>(integer(a[3]));
    f_rope = reinterpret_cast<decltype(f_rope)>(integer(a[4]));
    f_append = reinterpret_cast<decltype(f_append)>(integer(a[5]));
    f_logits = reinterpret_cast<decltype(f_logits)>(integer(a[6]));
    f_counts = reinterpret_cast<decltype(f_counts)>(integer(a[7]));
    f_prefix = reinterpret_cast<decltype(f_prefix)>(integer(a[8]));
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
                         method<prefix_attention>("prefix_attention"),
                         method<rope>("rope"),
                         method<cache_append>("cache_append"),
                         method<logits_adjust>("logits_adjust"),
                         method<token_counts>("token_counts"),
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
