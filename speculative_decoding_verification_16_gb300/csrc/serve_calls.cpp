// serve_calls.cpp -- Python calls of the paged serving operators
// (include/spec_verify_serve.h): argument checks and marshalling.
//
// A server issues these operators once a step or once a layer, and the smallest
// take a few microseconds on the GPU; checking and converting 10 to 25 arguments
// in Python and ctypes took 13 to 24 us a call.  The module has one function an
// operator: tensors and numbers by position, None where left out; it raises
// TypeError and ValueError for what the operator does not take and returns the
// C entry point's status.  No C++ exception leaves it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "spec_verify_serve.h"

namespace {

struct BadType : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct BadValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw BadType(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

void on_device(const at::Tensor& t, const char* name, at::Device d) {
  if (t.device() != d)
    throw BadValue(std::string(name) + " is on " + t.device().str() + ", expected " + d.str());
}

void of_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    throw BadType(std::string(name) + " must be " + c10::toString(type) + ", got " +
                  c10::toString(t.scalar_type()));
}

// Address of a contiguous tensor of this type and shape; nullptr for None.
void* flat(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
           at::Device d) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  of_type(t, name, type);
  const at::IntArrayRef want(shape);
  if (t.sizes() != want || !t.is_contiguous())
    throw BadValue(std::string(name) + " must be a contiguous tensor of shape " + shape_text(want) +
                   ", got " + shape_text(t.sizes()));
  on_device(t, name, d);
  return t.data_ptr();
}

int32_t dtype_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SV_BF16;
  if (t.scalar_type() == at::kFloat) return SV_FP32;
  throw BadType(std::string(name) + " must be bfloat16 or float32, got " +
                c10::toString(t.scalar_type()));
}

int32_t small(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) throw BadValue(std::string(name) + " is too large");
  return static_cast<int32_t>(v);
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadType(std::string(name) + " must be an integer");
  }
  return v;
}

// [rows, V] with contiguous rows: their stride.
int64_t row_stride(const at::Tensor& t, const char* name) {
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    throw BadValue(std::string(name) + " must have two dimensions and contiguous rows");
  return t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.stride(0), t.size(1));
}

// [rows, heads, head_dim] with a contiguous last dimension.
void rows_of_heads(const at::Tensor& t, const char* name, at::ScalarType type, at::Device d) {
  if (t.dim() != 3 || (t.size(2) > 1 && t.stride(2) != 1))
    throw BadValue(std::string(name) +
                   " must be [rows, heads, head_dim] with a contiguous last dimension");
  of_type(t, name, type);
  on_device(t, name, d);
}

void caches(const at::Tensor& k, const at::Tensor& v, int64_t head_dim, at::ScalarType type,
            at::Device d) {
  const at::Tensor* both[2] = {&k, &v};
  const char* names[2] = {"key_cache", "value_cache"};
  for (int i = 0; i < 2; ++i) {
    of_type(*both[i], names[i], type);
    if (both[i]->dim() != 4 || (head_dim > 1 && both[i]->stride(3) != 1))
      throw BadValue(std::string(names[i]) +
                     " must be [num_blocks, page_size, kv_heads, head_dim] with a contiguous last "
                     "dimension");
    on_device(*both[i], names[i], d);
  }
  if (k.sizes() != v.sizes() || k.strides() != v.strides())
    throw BadValue("key_cache and value_cache must have the same shape and strides");
  if (k.size(3) != head_dim)
    throw BadValue("the caches' head_dim is " + std::to_string(k.size(3)) + ", expected " +
                   std::to_string(head_dim));
}

int32_t cache_code(const at::Tensor& t, const char* name) {
  return t.scalar_type() == at::kFloat8_e4m3fn ? SV_E4M3 : dtype_code(t, name);
}

// Exponents of a pair of caches: int8, the caches' shape without its last dimension;
// both None where the caches are not of 8 bits.
struct Exponents {
  int8_t *k = nullptr, *v = nullptr;
  int64_t stride[4] = {0, 0, 0, 0};  // layer (0 without layers), block, token, head
};
Exponents exponents(PyObject* ko, PyObject* vo, const at::Tensor& cache) {
  Exponents e;
  if (cache.scalar_type() != at::kFloat8_e4m3fn) {
    if (ko != Py_None || vo != Py_None)
      throw BadType("key_exps and value_exps belong to caches of float8_e4m3fn");
    return e;
  }
  if (ko == Py_None || vo == Py_None)
    throw BadValue("caches of float8_e4m3fn need key_exps and value_exps");
  const at::Tensor *both[2] = {&tensor(ko, "key_exps"), &tensor(vo, "value_exps")};
  const char* names[2] = {"key_exps", "value_exps"};
  const at::IntArrayRef want = cache.sizes().slice(0, cache.dim() - 1);
  for (int i = 0; i < 2; ++i) {
    of_type(*both[i], names[i], at::kChar);
    on_device(*both[i], names[i], cache.device());
    if (both[i]->sizes() != want)
      throw BadValue(std::string(names[i]) + " must have shape " + shape_text(want) + ", got " +
                     shape_text(both[i]->sizes()));
  }
  if (both[0]->strides() != both[1]->strides())
    throw BadValue("key_exps and value_exps must have the same strides");
  e.k = static_cast<int8_t*>(both[0]->data_ptr()), e.v = static_cast<int8_t*>(both[1]->data_ptr());
  const int64_t n = both[0]->dim();
  for (int64_t i = 0; i < n; ++i) e.stride[4 - n + i] = both[0]->stride(i);
  return e;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadType(std::string(name) + " must be a number");
  }
  return v;
}

// The stream (an int, or None for the device's current one), with the tensors'
// device current while this lives.
struct Launch {
  int before = -1;
  void* stream;
  Launch(PyObject* o, at::Device d) {
    if (!d.is_cuda()) throw BadValue("tensors must be on a CUDA device, got " + d.str());
    stream = o == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(d.index()).stream())
                          : reinterpret_cast<void*>(integer(o, "stream"));
    // last: what throws above leaves no device to put back
    const int now = c10::cuda::current_device();
    if (now != d.index()) {
      c10::cuda::set_device(d.index());
      before = now;
    }
  }
  ~Launch() {
    if (before >= 0) c10::cuda::set_device(static_cast<c10::DeviceIndex>(before));
  }
};

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const BadType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// logits, uniforms, temperature, top_k, top_p, min_p, out_tokens, out_probs,
// dev_error, stream
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor& x = tensor(a[0], "logits");
    const int64_t stride = row_stride(x, "logits"), N = x.size(0), V = x.size(1);
    const int32_t type = dtype_code(x, "logits");
    const at::Device d = x.device();
    void* u = flat(a[1], "uniforms", at::kFloat, {N}, d);
    void* temperature = flat(a[2], "temperature", at::kFloat, {N}, d);
    void* top_k = flat(a[3], "top_k", at::kInt, {N}, d);
    void* top_p = flat(a[4], "top_p", at::kFloat, {N}, d);
    void* min_p = flat(a[5], "min_p", at::kFloat, {N}, d);
    void* tokens = flat(a[6], "out_tokens", at::kInt, {N}, d);
    void* probs = flat(a[7], "out_probs", at::kFloat, {N}, d);
    void* err = flat(a[8], "dev_error", at::kInt, {1}, d);
    const Launch at(a[9], d);
    return spec_verify_sample(x.data_ptr(), stride, small(N, "N"), small(V, "V"), type,
                              static_cast<float*>(temperature), static_cast<int32_t*>(top_k),
                              static_cast<float*>(top_p), static_cast<float*>(min_p),
                              static_cast<float*>(u), static_cast<int32_t*>(tokens),
                              static_cast<float*>(probs), static_cast<int32_t*>(err), at.stream);
  });
}

// context_lens, verify_lens, block_table, held, free_list, free_count, page_size,
// n_rows, row_offsets, seq_lens, positions, slots, held_out, free_count_out,
// dev_error, stream
PyObject* slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const at::Tensor& table = tensor(a[2], "block_table");
    const int64_t stride = row_stride(table, "block_table"), B = table.size(0);
    of_type(table, "block_table", at::kInt);
    const at::Device d = table.device();
    const int64_t rows = integer(a[7], "n_rows"), cap = tensor(a[4], "free_list").numel();
    auto i32 = [&](int i, const char* name, std::initializer_list<int64_t> shape) {
      return static_cast<int32_t*>(flat(a[i], name, at::kInt, shape, d));
    };
    int32_t* ctx = i32(0, "context_lens", {B});
    int32_t* fresh = i32(1, "verify_lens", {B});
    int32_t* held = i32(3, "held", {B});
    int32_t* list = i32(4, "free_list", {cap});
    int32_t* count = i32(5, "free_count", {1});
    int32_t* offsets = i32(8, "row_offsets", {B + 1});
    int32_t* seq = i32(9, "seq_lens", {B});
    int32_t* positions = i32(10, "positions", {rows});
    void* out = flat(a[11], "slots", at::kLong, {rows}, d);
    int32_t* held_out = i32(12, "held_out", {B});
    int32_t* count_out = i32(13, "free_count_out", {1});
    int32_t* err = i32(14, "dev_error", {1});
    const Launch at(a[15], d);
    return spec_verify_slots(ctx, fresh, small(B, "B"), small(integer(a[6], "page_size"), "page_size"),
                             static_cast<int32_t*>(table.data_ptr()), stride,
                             small(table.size(1), "width"), held, list, small(cap, "free_list"), count,
                             small(rows, "n_rows"), offsets, seq, positions,
                             static_cast<int64_t*>(out), held_out, count_out, err, at.stream);
  });
}

// key, value, slots, key_cache, value_cache, dev_error, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor &k = tensor(a[0], "key"), &v = tensor(a[1], "value"),
                     &kc = tensor(a[3], "key_cache"), &vc = tensor(a[4], "value_cache");
    const int32_t type = dtype_code(kc, "key_cache");
    const at::Device d = kc.device();
    rows_of_heads(k, "key", kc.scalar_type(), d);
    rows_of_heads(v, "value", kc.scalar_type(), d);
    if (k.sizes() != v.sizes()) throw BadValue("key and value must have the same shape");
    caches(kc, vc, k.size(2), kc.scalar_type(), d);
    if (kc.size(2) != k.size(1))
      throw BadValue("the caches hold " + std::to_string(kc.size(2)) + " heads, expected " +
                     std::to_string(k.size(1)));
    void* at_slots = flat(a[2], "slots", at::kLong, {k.size(0)}, d);
    void* err = flat(a[5], "dev_error", at::kInt, {1}, d);
    const Launch at(a[6], d);
    return spec_verify_append(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0),
                              v.stride(1), static_cast<int64_t*>(at_slots), small(k.size(0), "n_rows"),
                              small(k.size(1), "kv_heads"), small(k.size(2), "head_dim"), kc.data_ptr(),
                              vc.data_ptr(), kc.stride(0), kc.stride(1), kc.stride(2),
                              small(kc.size(0), "num_blocks"), small(kc.size(1), "page_size"), type,
                              static_cast<int32_t*>(err), at.stream);
  });
}

// query, key_cache, value_cache, block_table, seq_lens, row_offsets, max_len,
// scale, window, out, lse, dev_error, workspace, stream
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const at::Tensor &q = tensor(a[0], "query"), &kc = tensor(a[1], "key_cache"),
                     &vc = tensor(a[2], "value_cache"), &table = tensor(a[3], "block_table"),
                     &out = tensor(a[9], "out"), &ws = tensor(a[12], "workspace");
    const int32_t type = dtype_code(q, "query");
    const at::Device d = q.device();
    rows_of_heads(q, "query", q.scalar_type(), d);
    caches(kc, vc, q.size(2), q.scalar_type(), d);
    const int64_t stride = row_stride(table, "block_table"), B = table.size(0);
    of_type(table, "block_table", at::kInt);
    on_device(table, "block_table", d);
    rows_of_heads(out, "out", q.scalar_type(), d);
    if (out.sizes() != q.sizes()) throw BadValue("out must have the query's shape");
    void* seq = flat(a[4], "seq_lens", at::kInt, {B}, d);
    void* offsets = flat(a[5], "row_offsets", at::kInt, {B + 1}, d);
    void* lse = flat(a[10], "lse", at::kFloat, {q.size(0), q.size(1)}, d);
    void* err = flat(a[11], "dev_error", at::kInt, {1}, d);
    on_device(ws, "workspace", d);
    if (!ws.is_contiguous()) throw BadValue("workspace must be contiguous");
    const double scale = number(a[7], "scale");
    const Launch at(a[13], d);
    return spec_verify_attention(
        q.data_ptr(), q.stride(0), q.stride(1), kc.data_ptr(), vc.data_ptr(), kc.stride(0),
        kc.stride(1), kc.stride(2), static_cast<int32_t*>(table.data_ptr()), stride,
        small(table.size(1), "table_width"), static_cast<int32_t*>(seq), static_cast<int32_t*>(offsets),
        small(B, "B"), small(q.size(0), "n_rows"), small(integer(a[6], "max_len"), "max_len"),
        small(q.size(1), "heads"), small(kc.size(2), "kv_heads"), small(q.size(2), "head_dim"),
        small(kc.size(0), "num_blocks"), small(kc.size(1), "page_size"), type,
        static_cast<float>(scale), small(integer(a[8], "window"), "window"), out.data_ptr(),
        out.stride(0), out.stride(1), static_cast<float*>(lse), static_cast<int32_t*>(err),
        ws.data_ptr(), ws.numel() * ws.element_size(), at.stream);
  });
}

// Positions and frequencies of a rotation of `rows` rows: rotary_dim.
struct Rotation {
  const int32_t* positions = nullptr;
  const int64_t* freqs = nullptr;
  int32_t dim = 0, interleaved = 0;
  float amplitude = 1.0f;
};
Rotation rotation(PyObject* positions, PyObject* freqs, PyObject* interleaved, PyObject* amplitude,
                  int64_t rows, at::Device d) {
  Rotation r;
  if (freqs != Py_None) {
    const int64_t n = tensor(freqs, "freqs").numel();
    r.freqs = static_cast<int64_t*>(flat(freqs, "freqs", at::kLong, {n}, d));
    r.dim = small(2 * n, "freqs");
    if (positions == Py_None) throw BadValue("positions are needed where freqs are given");
    r.positions = static_cast<int32_t*>(flat(positions, "positions", at::kInt, {rows}, d));
  }
  r.interleaved = PyObject_IsTrue(interleaved);
  if (r.interleaved < 0) {
    PyErr_Clear();
    throw BadType("interleaved must be true or false");
  }
  r.amplitude = static_cast<float>(number(amplitude, "amplitude"));
  return r;
}

// x, positions, freqs, interleaved, amplitude, out, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &out = tensor(a[5], "out");
    const int32_t type = dtype_code(x, "x");
    const at::Device d = x.device();
    rows_of_heads(x, "x", x.scalar_type(), d);
    rows_of_heads(out, "out", x.scalar_type(), d);
    if (out.sizes() != x.sizes()) throw BadValue("out must have the shape of x");
    const Rotation r = rotation(a[1], a[2], a[3], a[4], x.size(0), d);
    const Launch at(a[6], d);
    return spec_verify_rope(x.data_ptr(), x.stride(0), x.stride(1), small(x.size(0), "n_rows"),
                            small(x.size(1), "heads"), small(x.size(2), "head_dim"), type,
                            r.positions, r.freqs, r.dim, r.interleaved, r.amplitude, out.data_ptr(),
                            out.stride(0), out.stride(1), at.stream);
  });
}

// query, key, value, positions, freqs, slots, key_cache, value_cache, interleaved,
// amplitude, key_exps, value_exps, out_query, dev_error, stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const at::Tensor &k = tensor(a[1], "key"), &v = tensor(a[2], "value"),
                     &kc = tensor(a[6], "key_cache"), &vc = tensor(a[7], "value_cache");
    const int32_t type = dtype_code(k, "key"), cache_type = cache_code(kc, "key_cache");
    const at::Device d = kc.device();
    rows_of_heads(k, "key", k.scalar_type(), d);
    rows_of_heads(v, "value", k.scalar_type(), d);
    if (k.sizes() != v.sizes()) throw BadValue("key and value must have the same shape");
    if (cache_type != SV_E4M3) of_type(kc, "key_cache", k.scalar_type());
    caches(kc, vc, k.size(2), kc.scalar_type(), d);
    if (kc.size(2) != k.size(1))
      throw BadValue("the caches hold " + std::to_string(kc.size(2)) + " heads, expected " +
                     std::to_string(k.size(1)));
    const Exponents e = exponents(a[10], a[11], kc);
    const Rotation r = rotation(a[3], a[4], a[8], a[9], k.size(0), d);
    void* at_slots = flat(a[5], "slots", at::kLong, {k.size(0)}, d);
    void* err = flat(a[13], "dev_error", at::kInt, {1}, d);
    const void* query = nullptr;
    void* out = nullptr;
    int64_t heads = 0, q[2] = {0, 0}, o[2] = {0, 0};
    if (a[0] != Py_None) {
      const at::Tensor &x = tensor(a[0], "query"), &y = tensor(a[12], "out_query");
      rows_of_heads(x, "query", k.scalar_type(), d);
      rows_of_heads(y, "out_query", k.scalar_type(), d);
      if (x.size(0) != k.size(0) || x.size(2) != k.size(2))
        throw BadValue("query must have the rows and the head_dim of key");
      if (x.sizes() != y.sizes()) throw BadValue("out_query must have the query's shape");
      query = x.data_ptr(), out = y.data_ptr(), heads = x.size(1);
      q[0] = x.stride(0), q[1] = x.stride(1), o[0] = y.stride(0), o[1] = y.stride(1);
    }
    const Launch at(a[14], d);
    return spec_verify_rope_append(
        query, q[0], q[1], small(heads, "heads"), k.data_ptr(), v.data_ptr(), k.stride(0),
        k.stride(1), v.stride(0), v.stride(1), small(k.size(1), "kv_heads"),
        small(k.size(0), "n_rows"), small(k.size(2), "head_dim"), type, r.positions, r.freqs, r.dim,
        r.interleaved, r.amplitude, out, o[0], o[1], static_cast<int64_t*>(at_slots),
        kc.data_ptr(), vc.data_ptr(), kc.stride(0), kc.stride(1), kc.stride(2),
        small(kc.size(0), "num_blocks"), small(kc.size(1), "page_size"), cache_type, e.k, e.v,
        e.stride[1], e.stride[2], e.stride[3], static_cast<int32_t*>(err), at.stream);
  });
}

// query, key_cache, value_cache, block_table, seq_lens, row_offsets, max_len, scale,
// window, key_exps, value_exps, tree_mask, positions, out, lse, dev_error, workspace,
// stream
PyObject* attention_ext(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&] {
    const at::Tensor &q = tensor(a[0], "query"), &kc = tensor(a[1], "key_cache"),
                     &vc = tensor(a[2], "value_cache"), &table = tensor(a[3], "block_table"),
                     &out = tensor(a[13], "out"), &ws = tensor(a[16], "workspace");
    const int32_t type = dtype_code(q, "query"), cache_type = cache_code(kc, "key_cache");
    const at::Device d = q.device();
    rows_of_heads(q, "query", q.scalar_type(), d);
    if (cache_type != SV_E4M3) of_type(kc, "key_cache", q.scalar_type());
    else of_type(q, "query", at::kBFloat16);
    caches(kc, vc, q.size(2), kc.scalar_type(), d);
    const Exponents e = exponents(a[9], a[10], kc);
    const int64_t stride = row_stride(table, "block_table"), B = table.size(0);
    of_type(table, "block_table", at::kInt);
    on_device(table, "block_table", d);
    rows_of_heads(out, "out", q.scalar_type(), d);
    if (out.sizes() != q.sizes()) throw BadValue("out must have the query's shape");
    void* seq = flat(a[4], "seq_lens", at::kInt, {B}, d);
    void* offsets = flat(a[5], "row_offsets", at::kInt, {B + 1}, d);
    void *mask = nullptr, *positions = nullptr;
    int64_t words = 0;
    if (a[11] != Py_None) {
      const at::Tensor& m = tensor(a[11], "tree_mask");
      if (m.dim() != 2) throw BadValue("tree_mask must have two dimensions");
      words = m.size(1);
      mask = flat(a[11], "tree_mask", at::kInt, {q.size(0), words}, d);
      positions = flat(a[12], "positions", at::kInt, {q.size(0)}, d);
    }
    void* lse = flat(a[14], "lse", at::kFloat, {q.size(0), q.size(1)}, d);
    void* err = flat(a[15], "dev_error", at::kInt, {1}, d);
    on_device(ws, "workspace", d);
    if (!ws.is_contiguous()) throw BadValue("workspace must be contiguous");
    const double scale = number(a[7], "scale");
    const Launch at(a[17], d);
    return spec_verify_attention_ext(
        q.data_ptr(), q.stride(0), q.stride(1), kc.data_ptr(), vc.data_ptr(), kc.stride(0),
        kc.stride(1), kc.stride(2), cache_type, e.k, e.v, e.stride[1], e.stride[2], e.stride[3],
        static_cast<int32_t*>(table.data_ptr()), stride, small(table.size(1), "table_width"),
        static_cast<int32_t*>(seq), static_cast<int32_t*>(offsets), static_cast<int32_t*>(mask),
        small(words, "mask_words"), static_cast<int32_t*>(positions), small(B, "B"),
        small(q.size(0), "n_rows"), small(integer(a[6], "max_len"), "max_len"),
        small(q.size(1), "heads"), small(kc.size(2), "kv_heads"), small(q.size(2), "head_dim"),
        small(kc.size(0), "num_blocks"), small(kc.size(1), "page_size"), type,
        static_cast<float>(scale), small(integer(a[8], "window"), "window"), out.data_ptr(),
        out.stride(0), out.stride(1), static_cast<float*>(lse), static_cast<int32_t*>(err),
        ws.data_ptr(), ws.numel() * ws.element_size(), at.stream);
  });
}

// A contiguous int32 row per token, and the requests' offsets: rows and requests.
struct TreeRows {
  int64_t rows, B;
  at::Device d;
};
TreeRows tree_rows(PyObject* row, const char* name, PyObject* offsets) {
  const at::Tensor &t = tensor(row, name), &o = tensor(offsets, "row_offsets");
  if (o.numel() < 2) throw BadValue("row_offsets must have B + 1 entries");
  return {t.dim() > 0 ? t.size(0) : 0, o.numel() - 1, t.device()};
}

// parents, seq_lens, row_offsets, max_len, positions, mask, dev_error, stream
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const TreeRows r = tree_rows(a[0], "parents", a[2]);
    const at::Tensor& m = tensor(a[5], "mask");
    if (m.dim() != 2) throw BadValue("mask must have two dimensions");
    auto i32 = [&](int i, const char* name, std::initializer_list<int64_t> shape) {
      return static_cast<int32_t*>(flat(a[i], name, at::kInt, shape, r.d));
    };
    int32_t* parents = i32(0, "parents", {r.rows});
    int32_t* seq = i32(1, "seq_lens", {r.B});
    int32_t* offsets = i32(2, "row_offsets", {r.B + 1});
    int32_t* positions = i32(4, "positions", {r.rows});
    int32_t* mask = i32(5, "mask", {r.rows, m.size(1)});
    int32_t* err = i32(6, "dev_error", {1});
    const Launch at(a[7], r.d);
    return spec_verify_tree(parents, seq, offsets, small(r.B, "B"), small(r.rows, "n_rows"),
                            small(integer(a[3], "max_len"), "max_len"), positions, mask,
                            small(m.size(1), "mask_words"), err, at.stream);
  });
}

// tokens, next_tokens, parents, row_offsets, max_len, out_tokens, path, accept_len,
// dev_error, stream
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const TreeRows r = tree_rows(a[0], "tokens", a[3]);
    auto i32 = [&](int i, const char* name, int64_t count) {
      return static_cast<int32_t*>(flat(a[i], name, at::kInt, {count}, r.d));
    };
    int32_t* tokens = i32(0, "tokens", r.rows);
    int32_t* next = i32(1, "next_tokens", r.rows);
    int32_t* parents = i32(2, "parents", r.rows);
    int32_t* offsets = i32(3, "row_offsets", r.B + 1);
    int32_t* out = i32(5, "out_tokens", r.rows);
    int32_t* path = i32(6, "path", r.rows);
    int32_t* len = i32(7, "accept_len", r.B);
    int32_t* err = i32(8, "dev_error", 1);
    const Launch at(a[9], r.d);
    return spec_verify_tree_accept(tokens, next, parents, offsets, small(r.B, "B"),
                                   small(r.rows, "n_rows"),
                                   small(integer(a[4], "max_len"), "max_len"), out, path, len, err,
                                   at.stream);
  });
}

// path, accept_len, row_offsets, slots, key_cache, value_cache, max_len, key_exps,
// value_exps, dev_error, stream
PyObject* tree_move(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const TreeRows r = tree_rows(a[0], "path", a[2]);
    const at::Tensor &kc = tensor(a[4], "key_cache"), &vc = tensor(a[5], "value_cache");
    const int32_t cache_type = cache_code(kc, "key_cache");
    const int64_t nd = kc.dim(), layers = nd == 5 ? kc.size(0) : 1, l = nd == 5 ? 1 : 0;
    if ((nd != 4 && nd != 5) || (kc.size(nd - 1) > 1 && kc.stride(nd - 1) != 1))
      throw BadValue("caches must be [num_blocks, page_size, kv_heads, head_dim], with layers "
                     "before them or not, and a contiguous last dimension");
    of_type(vc, "value_cache", kc.scalar_type());
    on_device(kc, "key_cache", r.d);
    on_device(vc, "value_cache", r.d);
    if (kc.sizes() != vc.sizes() || kc.strides() != vc.strides())
      throw BadValue("key_cache and value_cache must have the same shape and strides");
    const Exponents e = exponents(a[7], a[8], kc);
    void* path = flat(a[0], "path", at::kInt, {r.rows}, r.d);
    void* len = flat(a[1], "accept_len", at::kInt, {r.B}, r.d);
    void* offsets = flat(a[2], "row_offsets", at::kInt, {r.B + 1}, r.d);
    void* at_slots = flat(a[3], "slots", at::kLong, {r.rows}, r.d);
    void* err = flat(a[9], "dev_error", at::kInt, {1}, r.d);
    const Launch at(a[10], r.d);
    return spec_verify_tree_move(
        static_cast<int32_t*>(path), static_cast<int32_t*>(len), static_cast<int32_t*>(offsets),
        static_cast<int64_t*>(at_slots), small(r.B, "B"), small(r.rows, "n_rows"),
        small(integer(a[6], "max_len"), "max_len"), small(layers, "layers"),
        small(kc.size(l + 2), "kv_heads"), small(kc.size(l + 3), "head_dim"), kc.data_ptr(),
        vc.data_ptr(), l != 0 ? kc.stride(0) : 0, kc.stride(l), kc.stride(l + 1), kc.stride(l + 2),
        small(kc.size(l), "num_blocks"), small(kc.size(l + 1), "page_size"), cache_type, e.k, e.v,
        e.stride[0], e.stride[1], e.stride[2], e.stride[3], static_cast<int32_t*>(err), at.stream);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<sample>("sample"), method<slots>("slots"), method<append>("append"),
                         method<attention>("attention"), method<rope>("rope"),
                         method<rope_append>("rope_append"),
                         method<attention_ext>("attention_ext"), method<tree>("tree"),
                         method<tree_accept>("tree_accept"), method<tree_move>("tree_move"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_calls() { return PyModule_Create(&module); }
