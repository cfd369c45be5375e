// gdn_binding.cpp -- argument marshalling of the calls that take a few microseconds on the GPU: torch tensors in, addresses and
// sizes out, in C++ instead of Python attribute by attribute (a call with six tensors spent 4 us of the host's time on that, 8 us
// in all, next to 2 us of GPU time). It knows nothing of the library but the addresses of its C entry points, which the Python
// binding hands over once (bind). Every function returns the call's gdn_status; what is not a tensor of the right type, shape
// or device raises ValueError before the call.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "gdn.h"

namespace {

struct Entries {
  decltype(&gdn_rope) rope = nullptr;
  decltype(&gdn_cache4_append) append = nullptr;
  decltype(&gdn_cache4_read) read = nullptr;
  decltype(&gdn_attn4_decode) decode = nullptr;
  decltype(&gdn_attn4_prefill) prefill = nullptr;
} entry;

struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int32_t small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " must fit in 32 bits");
  return static_cast<int32_t>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

// The checks of one call: all tensors on the current device.
struct Call {
  void on_device(const at::Tensor& t, const char* name) const {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a device tensor");
    if (t.device().index() != c10::cuda::current_device()) refuse(std::string(name) + " must be on the current device");
  }
  [[noreturn]] static void shape_error(const at::Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    std::ostringstream s;
    s << name << " must be " << type << " of shape " << at::IntArrayRef(shape) << ", not " << t.scalar_type() << " " << t.sizes();
    refuse(s.str());
  }
  static bool fits(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape);
  }
  // a dense tensor of this type and shape; null if it is empty
  void* dense(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(o, name);
    if (!fits(t, type, shape)) shape_error(t, name, type, shape);
    if (t.numel() == 0) return nullptr;
    on_device(t, name);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  // bf16 [tokens, heads, d] with dense heads: the address, and elements from one token to the next
  std::pair<void*, int64_t> tokens(PyObject* o, const char* name, int64_t n, int64_t heads, int64_t d) const {
    const at::Tensor& t = tensor(o, name);
    if (!fits(t, at::kBFloat16, {n, heads, d})) shape_error(t, name, at::kBFloat16, {n, heads, d});
    if (t.numel() == 0) return {nullptr, heads * d};
    on_device(t, name);
    if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && heads > 1)) refuse(std::string(name) + " must have dense heads");
    return {t.data_ptr(), n > 1 ? t.stride(0) : heads * d};  // (one token: its stride means nothing)
  }
  // any tensor in one piece, or None
  std::pair<void*, size_t> block(PyObject* o, const char* name) const {
    if (o == Py_None) return {nullptr, 0};
    const at::Tensor& t = tensor(o, name);
    if (t.numel() == 0) return {nullptr, 0};
    on_device(t, name);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return {t.data_ptr(), t.nbytes()};
  }
  int32_t* error_word(PyObject* o) const {
    if (o != Py_None && tensor(o, "err").scalar_type() != at::kInt) refuse("err must be int32");
    return static_cast<int32_t*>(block(o, "err").first);
  }
  static void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  }
};

// The 4-bit cache's arrays; its shape is the key array's.
struct Cache {
  void *k, *v;
  uint8_t *k_scale, *v_scale;
  int32_t blocks;
  gdn_cache_dims dims;
  Cache(const Call& c, PyObject* const* o, int64_t q_heads) {
    const at::Tensor& t = tensor(o[0], "k_cache");
    if (t.dim() != 4) refuse("k_cache must be [num_blocks, Hkv, block_size, head_dim / 2]");
    const int64_t n = t.size(0), h = t.size(1), bs = t.size(2), d = 2 * t.size(3);
    for (int64_t x : {n, h, bs, d, q_heads})
      if (x > INT32_MAX) refuse("the cache's sizes must fit in 32 bits");
    k = c.dense(o[0], "k_cache", at::kByte, {n, h, bs, d / 2});
    v = c.dense(o[1], "v_cache", at::kByte, {n, h, bs / 2, d});
    const at::ScalarType type = tensor(o[2], "k_scale").scalar_type();
    if (type != at::kByte && type != at::kFloat8_e8m0fnu) refuse("the scales must be float8_e8m0fnu (or its bytes)");
    k_scale = static_cast<uint8_t*>(c.dense(o[2], "k_scale", type, {n, h, bs, d / 32}));
    v_scale = static_cast<uint8_t*>(c.dense(o[3], "v_scale", type, {n, h, bs, d / 32}));
    blocks = static_cast<int32_t>(n);
    dims = {static_cast<int32_t>(q_heads), static_cast<int32_t>(h), static_cast<int32_t>(d), static_cast<int32_t>(bs)};
  }
};

int64_t size_of(PyObject* o, const char* name, int64_t dim, int64_t i) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dim) refuse(std::string(name) + " must have " + std::to_string(dim) + " dimensions");
  if (t.size(i) > INT32_MAX) refuse(std::string(name) + " must have sizes that fit in 32 bits");
  return t.size(i);
}

// q, k, positions, q_out, k_out, turns, rot_dim, factor, layout, stream
gdn_status rope(PyObject* const* a) {
  const Call c{};
  const int64_t n = size_of(a[0], "q", 3, 0), hq = size_of(a[0], "q", 3, 1), d = size_of(a[0], "q", 3, 2);
  const bool keys = a[1] != Py_None;
  if (!keys && a[4] != Py_None) refuse("k_out without k: nothing would be written to it");
  const int64_t h = keys ? size_of(a[1], "k", 3, 1) : 0;
  const int32_t rot = small(a[6], "rot_dim");
  const auto q = c.tokens(a[0], "q", n, hq, d), q_out = c.tokens(a[3], "q_out", n, hq, d);
  std::pair<void*, int64_t> k{nullptr, 0}, k_out{nullptr, 0};
  if (keys) {
    k = c.tokens(a[1], "k", n, h, d);
    k_out = c.tokens(a[4], "k_out", n, h, d);
  }
  const void* pos = c.dense(a[2], "positions", at::kInt, {n});
  const void* turns = c.dense(a[5], "rope.turns", at::kLong, {rot / 2});
  return entry.rope(q.first, q.second, k.first, k.second, static_cast<const int32_t*>(pos), static_cast<int32_t>(n),
                    static_cast<int32_t>(hq), static_cast<int32_t>(h), static_cast<int32_t>(d), rot,
                    static_cast<gdn_rope_layout>(small(a[8], "layout")), static_cast<const uint64_t*>(turns), real(a[7]), q_out.first,
                    q_out.second, k_out.first, k_out.second, Call::stream(a[9]));
}

// k, v, slot_map, cache (4), err, stream
gdn_status append(PyObject* const* a) {
  const Call c{};
  const Cache cache(c, a + 3, 1);
  const int64_t n = size_of(a[2], "slot_map", 1, 0);
  const auto k = c.tokens(a[0], "k", n, cache.dims.num_kv_heads, cache.dims.head_dim), v = c.tokens(a[1], "v", n, cache.dims.num_kv_heads, cache.dims.head_dim);
  const void* slots = c.dense(a[2], "slot_map", at::kInt, {n});
  return entry.append(k.first, k.second, v.first, v.second, static_cast<const int32_t*>(slots), static_cast<int32_t>(n), cache.k, cache.v,
                      cache.k_scale, cache.v_scale, cache.blocks, cache.dims, c.error_word(a[7]), Call::stream(a[8]));
}

// cache (4), slot_map, k, v, err, stream
gdn_status read(PyObject* const* a) {
  const Call c{};
  const Cache cache(c, a, 1);
  const int64_t n = size_of(a[4], "slot_map", 1, 0);
  const auto k = c.tokens(a[5], "k", n, cache.dims.num_kv_heads, cache.dims.head_dim), v = c.tokens(a[6], "v", n, cache.dims.num_kv_heads, cache.dims.head_dim);
  const void* slots = c.dense(a[4], "slot_map", at::kInt, {n});
  return entry.read(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.blocks, static_cast<const int32_t*>(slots), static_cast<int32_t>(n),
                    cache.dims, k.first, k.second, v.first, v.second, c.error_word(a[7]), Call::stream(a[8]));
}

// What both attention calls take: q, cache (4), block_table, lens, out, workspace, scale (None: head_dim ** -0.5), err, stream
struct Attention {
  const Call c{};
  const int64_t n, hq;
  const Cache cache;
  const std::pair<void*, int64_t> q;
  const int64_t batch, width;
  const int32_t *table, *lens;
  void* out;
  const std::pair<void*, size_t> workspace;
  const float scale;
  int32_t* err;
  void* stream;
  explicit Attention(PyObject* const* a)
      : n(size_of(a[0], "q", 3, 0)),
        hq(size_of(a[0], "q", 3, 1)),
        cache(c, a + 1, hq),
        q(c.tokens(a[0], "q", n, hq, cache.dims.head_dim)),
        batch(size_of(a[6], "lens", 1, 0)),
        width(size_of(a[5], "block_table", 2, 1)),
        table(static_cast<const int32_t*>(c.dense(a[5], "block_table", at::kInt, {batch, width}))),
        lens(static_cast<const int32_t*>(c.dense(a[6], "lens", at::kInt, {batch}))),
        out(c.dense(a[7], "out", at::kBFloat16, {n, hq, cache.dims.head_dim})),
        workspace(c.block(a[8], "workspace")),
        scale(a[9] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(cache.dims.head_dim))) : real(a[9])),
        err(c.error_word(a[10])),
        stream(Call::stream(a[11])) {}
};

gdn_status decode(PyObject* const* a) {
  const Attention x(a);
  if (x.batch != x.n) refuse("lens must have an entry for each row of q");
  return entry.decode(x.q.first, x.q.second, x.cache.k, x.cache.v, x.cache.k_scale, x.cache.v_scale, x.cache.blocks, x.table,
                      static_cast<int32_t>(x.width), x.lens, static_cast<int32_t>(x.n), x.cache.dims, x.scale, x.out,
                      x.workspace.first, x.workspace.second, x.err, x.stream);
}

// ... cu_tokens, held_blocks (None: batch x width)
gdn_status prefill(PyObject* const* a) {
  const Attention x(a);
  const void* cu = x.c.dense(a[12], "cu_tokens", at::kInt, {x.batch + 1});
  const int64_t all = x.batch * x.width;
  const int32_t held = a[13] == Py_None ? static_cast<int32_t>(all < INT32_MAX ? all : INT32_MAX) : small(a[13], "held_blocks");
  return entry.prefill(x.q.first, x.q.second, static_cast<const int32_t*>(cu), x.cache.k, x.cache.v, x.cache.k_scale, x.cache.v_scale,
                       x.cache.blocks, x.table, static_cast<int32_t>(x.width), x.lens, static_cast<int32_t>(x.batch),
                       static_cast<int32_t>(x.n), held, x.cache.dims, x.scale, x.out, x.workspace.first, x.workspace.second, x.err,
                       x.stream);
}

template <gdn_status (*call)(PyObject* const*), int count>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, not %zd", count, n);
    return nullptr;
  }
  try {
    if (!entry.prefill) refuse("the library's entry points have not been bound");
    return PyLong_FromLong(call(args));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "an unknown error");
  }
  return nullptr;
}

// addresses of gdn_rope, gdn_cache4_append, gdn_cache4_read, gdn_attn4_decode, gdn_attn4_prefill
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "5 addresses expected");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  entry.rope = reinterpret_cast<decltype(entry.rope)>(p[0]);
  entry.append = reinterpret_cast<decltype(entry.append)>(p[1]);
  entry.read = reinterpret_cast<decltype(entry.read)>(p[2]);
  entry.decode = reinterpret_cast<decltype(entry.decode)>(p[3]);
  entry.prefill = reinterpret_cast<decltype(entry.prefill)>(p[4]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"rope", fast(method<rope, 10>), METH_FASTCALL, nullptr},
                         {"cache4_append", fast(method<append, 9>), METH_FASTCALL, nullptr},
                         {"cache4_read", fast(method<read, 9>), METH_FASTCALL, nullptr},
                         {"attn4_decode", fast(method<decode, 12>), METH_FASTCALL, nullptr},
                         {"attn4_prefill", fast(method<prefill, 14>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling of libgdn.so's calls.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
