// decode_ext.cpp -- the Python calls of the decode-step operators: checks of
// the tensors, allocation of the outputs on their stream, and the calls of
// include/moe_route.h.  Written against CPython and ATen because a decode step
// makes these calls once a layer on sizes where the host's time counts: the
// same checks cost ten times as much from Python.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/moe_route.h"

namespace {

using at::Tensor;

// A Python exception is set: unwinds to the entry point
struct Raised {};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised{};
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

std::string shape_text(c10::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v > INT32_MAX || v < INT32_MIN) refuse(std::string(name) + " does not fit 32 bits");
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

void on_device(const Tensor& t, const char* name, int dev) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != dev)
    refuse(std::string(name) + " must be on cuda:" + std::to_string(dev) + ", got " +
           t.device().str());
}

void of_type(const Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + type_name(type) + ", got " +
           type_name(t.scalar_type()));
}

// A contiguous vector of n elements
void* vec(const Tensor& t, at::ScalarType type, int64_t n, const char* name, int dev) {
  on_device(t, name, dev);
  of_type(t, type, name);
  if (t.dim() != 1 || t.size(0) != n) {
    std::ostringstream o;
    o << name << " must have shape (" << n << ",), got " << shape_text(t.sizes());
    refuse(o.str());
  }
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

void* optional_vec(PyObject* o, at::ScalarType type, int64_t n, const char* name, int dev) {
  return o == Py_None ? nullptr : vec(tensor(o, name), type, n, name, dev);
}

int64_t length(const Tensor& t, const char* name) {
  if (t.dim() != 1) refuse(std::string(name) + " must be a vector");
  return t.size(0);
}

uint32_t* error_word(PyObject* o, int dev) {
  return static_cast<uint32_t*>(optional_vec(o, at::kInt, 1, "err", dev));
}

struct Table {
  int32_t* p;
  int64_t width, stride;
};

Table block_table(const Tensor& t, int64_t rows, int dev) {
  on_device(t, "block_table", dev);
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows || t.size(1) < 1) {
    std::ostringstream o;
    o << "block_table must be torch.int32 [" << rows << ", max_pages], got "
      << type_name(t.scalar_type()) << " " << shape_text(t.sizes());
    refuse(o.str());
  }
  const int64_t width = t.size(1);
  if (rows > 0 && ((width > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < width)))
    refuse("block_table's rows must be contiguous and must not overlap");
  return {static_cast<int32_t*>(t.data_ptr()), width, rows > 1 ? t.stride(0) : width};
}

// Stride of axis i; one of a single element has none that matters
int64_t stride_of(const Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; }

void contiguous_last(const Tensor& t, const char* name) {
  const int64_t last = t.dim() - 1;
  if (t.size(last) > 1 && t.stride(last) != 1)
    refuse(std::string(name) + "'s vectors must be contiguous");
}

// [n, heads, head_dim] with contiguous vectors
void rows3(const Tensor& t, at::ScalarType type, int64_t n, int64_t heads, int64_t dim,
           const char* name, int dev) {
  on_device(t, name, dev);
  of_type(t, type, name);
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != dim) {
    std::ostringstream o;
    o << name << " must have shape (" << n << ", " << heads << ", " << dim << "), got "
      << shape_text(t.sizes());
    refuse(o.str());
  }
  contiguous_last(t, name);
}

// A cache whose vectors are only moved: scales do not matter
moe_kv_cache_t kv_cache(const Tensor& k, const Tensor& v, int dev) {
  on_device(k, "k_cache", dev);
  on_device(v, "v_cache", dev);
  moe_kv_cache_t c = {};
  switch (k.scalar_type()) {
    case at::kFloat: c.kv_dtype = MOE_KV_F32; break;
    case at::kBFloat16: c.kv_dtype = MOE_KV_BF16; break;
    case at::kFloat8_e4m3fn: c.kv_dtype = MOE_KV_E4M3; break;
    default:
      refuse(std::string("k_cache must be float32, bfloat16 or float8_e4m3fn, got ") +
             type_name(k.scalar_type()));
  }
  bool alike = v.scalar_type() == k.scalar_type() && k.dim() == 4 && v.sizes() == k.sizes();
  for (int i = 0; alike && i < 4; ++i) alike = stride_of(k, i) == stride_of(v, i);
  if (!alike)
    refuse(
        "k_cache and v_cache must be [num_pages, page_size, kv_heads, head_dim] of one type and "
        "the same strides");
  contiguous_last(k, "k_cache");
  for (int i = 0; i < 4; ++i)
    if (k.size(i) > INT32_MAX) refuse("k_cache's sizes must fit 32 bits");
  c.num_pages = static_cast<int32_t>(k.size(0));
  c.page_size = static_cast<int32_t>(k.size(1));
  c.kv_heads = static_cast<int32_t>(k.size(2));
  c.head_dim = static_cast<int32_t>(k.size(3));
  c.stride_page = stride_of(k, 0);
  c.stride_token = stride_of(k, 1);
  c.stride_head = stride_of(k, 2);
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  return c;
}

moe_kv_cache_t kv_cache(const Tensor& k, const Tensor& v, PyObject* k_scale, PyObject* v_scale,
                        int dev) {
  moe_kv_cache_t c = kv_cache(k, v, dev);
  const bool q8 = c.kv_dtype == MOE_KV_E4M3;
  if (q8 && (k_scale == Py_None || v_scale == Py_None))
    refuse("a float8_e4m3fn cache needs k_scale and v_scale");
  if (!q8 && (k_scale != Py_None || v_scale != Py_None))
    refuse("scales are only used by a float8_e4m3fn cache");
  c.k_scale = static_cast<const float*>(optional_vec(k_scale, at::kFloat, c.kv_heads, "k_scale", dev));
  c.v_scale = static_cast<const float*>(optional_vec(v_scale, at::kFloat, c.kv_heads, "v_scale", dev));
  return c;
}

// Where a call runs: the tensors' device, and the stream given (a handle) or
// the current one.  What the call allocates belongs to that stream.
struct Place {
  int dev;
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> on;
  void* stream;

  Place(const Tensor& t, const char* name, PyObject* given)
      : dev(cuda_index(t, name)), device(static_cast<c10::DeviceIndex>(dev)) {
    if (given == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
      return;
    }
    stream = PyLong_AsVoidPtr(given);
    if (!stream && PyErr_Occurred()) throw Raised{};
    on.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                static_cast<c10::DeviceIndex>(dev)));
  }
  static int cuda_index(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t.get_device();
  }
  Tensor make(c10::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions()
                                .dtype(type)
                                .device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
  }
};

void check(int rc, const char* what) {
  if (rc == MOE_OK) return;
  PyObject* m = PyImport_ImportModule("serving_moe_route_gb300._binding");
  if (m) {
    if (PyObject* e = PyObject_CallMethod(m, "MoeError", "is", rc, what)) {
      PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
      Py_DECREF(e);
    }
    Py_DECREF(m);
  }
  throw Raised{};
}

// Entry points: count the arguments, and let no C++ exception out
template <typename F>
PyObject* entry(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// n elements of a buffer, from `at` on, as a tensor of its own (of that type, the
// buffer's by default; `at` counts elements of it)
Tensor cut(const Tensor& buffer, int64_t at, int64_t n,
           at::ScalarType type = at::ScalarType::Undefined) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(buffer.storage()), buffer.key_set(),
      type == at::ScalarType::Undefined ? buffer.dtype() : c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// Tells autograd that a tensor of the caller's has been written, as an in-place
// operation does: a graph that saved it refuses to run backward through it
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

int32_t* i32(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// (ctx_lens, new_lens, block_table, free_pages, n_free, page_size, num_pages,
//  max_tokens, n_free_out, err, stream)
PyObject* kv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 11, [&] {
    const Tensor &ctx = tensor(a[0], "ctx_lens"), &nw = tensor(a[1], "new_lens"),
                 &table = tensor(a[2], "block_table"), &free = tensor(a[3], "free_pages"),
                 &left = tensor(a[4], "n_free");
    const Place at_(ctx, "ctx_lens", a[10]);
    const int dev = at_.dev;
    const int64_t B = length(ctx, "ctx_lens"), cap = length(free, "free_pages");
    void* const pc = vec(ctx, at::kInt, B, "ctx_lens", dev);
    void* const pn = vec(nw, at::kInt, B, "new_lens", dev);
    const Table t = block_table(table, B, dev);
    void* const pf = vec(free, at::kInt, cap, "free_pages", dev);
    void* const pl = vec(left, at::kInt, 1, "n_free", dev);
    const long long page = integer(a[5], "page_size"), pages = integer(a[6], "num_pages"),
                    tokens = integer(a[7], "max_tokens");
    if (tokens < 0) refuse("max_tokens must not be negative");
    if (B > INT32_MAX || cap > INT32_MAX || t.width > INT32_MAX) refuse("sizes must fit 32 bits");
    const Tensor all = at_.make({2 * tokens + 2 * B + 2}, at::kInt);
    const Tensor slots = cut(all, 0, tokens), positions = cut(all, tokens, tokens),
                 starts = cut(all, 2 * tokens, B + 1), lens = cut(all, 2 * tokens + B + 1, B);
    Tensor out;
    if (a[8] == Py_None) {
      out = cut(all, 2 * tokens + 2 * B + 1, 1);
    } else {
      out = tensor(a[8], "n_free_out");
      vec(out, at::kInt, 1, "n_free_out", dev);
    }
    check(moe_kv_step(static_cast<int32_t*>(pc), static_cast<int32_t*>(pn), static_cast<int>(B), t.p,
                      static_cast<int>(t.width), t.stride, static_cast<int32_t*>(pf),
                      static_cast<int>(cap), static_cast<int32_t*>(pl), i32(out),
                      static_cast<int>(pages), static_cast<int>(page), static_cast<int>(tokens),
                      i32(slots), i32(positions), i32(starts), i32(lens), error_word(a[9], dev),
                      at_.stream),
          "moe_kv_step");
    written(table);
    if (a[8] != Py_None) written(out);
    PyObject* r = PyTuple_New(5);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(slots));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(positions));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(starts));
    PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(lens));
    PyTuple_SET_ITEM(r, 4, THPVariable_Wrap(out));
    return r;
  });
}

// (done, block_table, free_pages, n_free, num_pages, err, stream)
PyObject* kv_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const Tensor &done = tensor(a[0], "done"), &table = tensor(a[1], "block_table"),
                 &free = tensor(a[2], "free_pages"), &left = tensor(a[3], "n_free");
    const Place at_(done, "done", a[6]);
    const int64_t B = length(done, "done"), cap = length(free, "free_pages");
    const Table t = block_table(table, B, at_.dev);
    if (B > INT32_MAX || cap > INT32_MAX || t.width > INT32_MAX) refuse("sizes must fit 32 bits");
    void* const pd = vec(done, at::kInt, B, "done", at_.dev);
    void* const pf = vec(free, at::kInt, cap, "free_pages", at_.dev);
    void* const pl = vec(left, at::kInt, 1, "n_free", at_.dev);
    check(moe_kv_release(static_cast<int32_t*>(pd), static_cast<int>(B), t.p,
                         static_cast<int>(t.width), t.stride, static_cast<int32_t*>(pf),
                         static_cast<int>(cap), static_cast<int32_t*>(pl),
                         static_cast<int>(integer(a[4], "num_pages")), error_word(a[5], at_.dev),
                         at_.stream),
          "moe_kv_release");
    written(table);
    written(free);
    written(left);
    Py_RETURN_NONE;
  });
}

at::ScalarType vector_type(const moe_kv_cache_t& c) {
  return c.kv_dtype == MOE_KV_F32 ? at::kFloat : at::kBFloat16;
}

// (k, v, slots, k_cache, v_cache, k_scale, v_scale, err, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&]() -> PyObject* {
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                 &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache");
    const Place at_(kc, "k_cache", a[8]);
    const moe_kv_cache_t c = kv_cache(kc, vc, a[5], a[6], at_.dev);
    const int64_t N = length(slots, "slots");
    if (N > INT32_MAX) refuse("slots must fit 32 bits");
    rows3(k, vector_type(c), N, c.kv_heads, c.head_dim, "k", at_.dev);
    rows3(v, vector_type(c), N, c.kv_heads, c.head_dim, "v", at_.dev);
    void* const ps = vec(slots, at::kInt, N, "slots", at_.dev);
    check(moe_kv_append(&c, k.data_ptr(), stride_of(k, 0), stride_of(k, 1), v.data_ptr(),
                        stride_of(v, 0), stride_of(v, 1), static_cast<int>(N),
                        static_cast<int32_t*>(ps), error_word(a[7], at_.dev), at_.stream),
          "moe_kv_append");
    written(kc);
    written(vc);
    Py_RETURN_NONE;
  });
}

// (q, k_cache, v_cache, block_table, seq_lens, scale, window, k_scale, v_scale,
//  out, return_lse, workspace, err, stream)
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 14, [&]() -> PyObject* {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"),
                 &vc = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table"),
                 &lens = tensor(a[4], "seq_lens");
    const Place at_(kc, "k_cache", a[13]);
    const int dev = at_.dev;
    const moe_kv_cache_t c = kv_cache(kc, vc, a[7], a[8], dev);
    if (q.dim() != 3) refuse("q must be [B, Hq, head_dim]");
    const int64_t B = q.size(0), hq = q.size(1), dim = c.head_dim;
    rows3(q, vector_type(c), B, hq, dim, "q", dev);
    if (hq < 1 || c.kv_heads < 1 || hq % c.kv_heads) {
      std::ostringstream o;
      o << "Hq=" << hq << " is not a multiple of kv_heads=" << c.kv_heads;
      refuse(o.str());
    }
    const Table t = block_table(table, B, dev);
    void* const pl = vec(lens, at::kInt, B, "seq_lens", dev);
    if (B > INT32_MAX || hq > INT32_MAX || t.width > INT32_MAX) refuse("sizes must fit 32 bits");
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(dim)) : number(a[5]);
    const long long window = integer(a[6], "window");
    Tensor out;
    if (a[9] == Py_None) {
      out = at_.make({B, hq, dim}, vector_type(c));
    } else {
      out = tensor(a[9], "out");
      rows3(out, vector_type(c), B, hq, dim, "out", dev);
    }
    const int with_lse = PyObject_IsTrue(a[10]);
    if (with_lse < 0) throw Raised{};
    Tensor lse;
    if (with_lse) lse = at_.make({B, hq}, at::kFloat);
    const size_t need = moe_attn_workspace(c.kv_dtype, c.head_dim);
    c10::DataPtr own;  // returned to the stream's pool when the call has been enqueued
    void* ws;
    size_t bytes = need;
    if (a[11] == Py_None) {
      own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
      ws = own.get();
    } else {
      const Tensor& w = tensor(a[11], "workspace");
      bytes = static_cast<size_t>(length(w, "workspace"));
      ws = vec(w, at::kByte, w.size(0), "workspace", dev);
    }
    check(moe_attn_decode(&c, q.data_ptr(), stride_of(q, 0), stride_of(q, 1), static_cast<int>(B),
                          static_cast<int>(hq), t.p, static_cast<int>(t.width), t.stride,
                          static_cast<int32_t*>(pl), static_cast<float>(scale),
                          static_cast<int>(window), out.data_ptr(), stride_of(out, 0),
                          stride_of(out, 1), with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                          ws, bytes, error_word(a[12], dev), at_.stream),
          "moe_attn_decode");
    if (a[9] != Py_None) written(out);
    if (!with_lse) return THPVariable_Wrap(out);
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
    return r;
  });
}

// (logits, u, temperature, top_k, top_p, min_p, stream)
PyObject* sample_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const Tensor &x = tensor(a[0], "logits"), &u = tensor(a[1], "u");
    const Place at_(x, "logits", a[6]);
    const int dev = at_.dev;
    if (x.scalar_type() != at::kFloat && x.scalar_type() != at::kBFloat16)
      refuse("logits must be float32 or bfloat16");
    if (x.dim() != 2 || x.size(1) < 1 || (x.size(1) > 1 && x.stride(1) != 1))
      refuse("logits must be [B, V] with contiguous rows");
    const int64_t B = x.size(0), V = x.size(1);
    void* const pu = vec(u, at::kFloat, B, "u", dev);
    void* const pt = optional_vec(a[2], at::kFloat, B, "temperature", dev);
    void* const pk = optional_vec(a[3], at::kInt, B, "top_k", dev);
    void* const pp = optional_vec(a[4], at::kFloat, B, "top_p", dev);
    void* const pm = optional_vec(a[5], at::kFloat, B, "min_p", dev);
    if (B > INT32_MAX || V > INT32_MAX) refuse("sizes must fit 32 bits");
    const Tensor ids = at_.make({B}, at::kInt), probs = at_.make({B}, at::kFloat);
    check(moe_sample(x.data_ptr(), x.scalar_type() == at::kFloat ? MOE_LOGITS_F32 : MOE_LOGITS_BF16,
                     static_cast<int>(B), static_cast<int>(V), B > 1 ? x.stride(0) : V,
                     static_cast<float*>(pu), static_cast<float*>(pt), static_cast<int32_t*>(pk),
                     static_cast<float*>(pp), static_cast<float*>(pm), i32(ids),
                     static_cast<float*>(probs.data_ptr()), at_.stream),
          "moe_sample");
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(ids));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(probs));
    return r;
  });
}

// A contiguous matrix of n rows; returns its width
int64_t matrix(const Tensor& t, at::ScalarType type, int64_t n, const char* name, int dev) {
  on_device(t, name, dev);
  of_type(t, type, name);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) > INT32_MAX) {
    std::ostringstream o;
    o << name << " must have shape (" << n << ", n), got " << shape_text(t.sizes());
    refuse(o.str());
  }
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.size(1);
}

// starts of B requests: B
int64_t requests_of(const Tensor& starts, int dev) {
  const int64_t n = length(starts, "starts");
  if (n < 1 || n - 1 > INT32_MAX) refuse("starts must hold one number more than there are requests");
  vec(starts, at::kInt, n, "starts", dev);
  return n - 1;
}

void fits(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + " must fit 32 bits");
}

long long nodes_of(PyObject* o, const char* name) {
  const long long n = integer(o, name);
  if (n < 1 || n > MOE_TREE_MAX)
    refuse(std::string(name) + " must be from 1 to " + std::to_string(MOE_TREE_MAX));
  return n;
}

// (parents, starts, seq_lens, max_new, err, stream)
PyObject* tree_masks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&]() -> PyObject* {
    const Tensor &parents = tensor(a[0], "parents"), &starts = tensor(a[1], "starts"),
                 &lens = tensor(a[2], "seq_lens");
    const Place at_(parents, "parents", a[5]);
    const int dev = at_.dev;
    const int64_t N = length(parents, "parents"), B = requests_of(starts, dev);
    fits(N, "parents");
    vec(parents, at::kInt, N, "parents", dev);
    vec(lens, at::kInt, B, "seq_lens", dev);
    const long long max_new = nodes_of(a[3], "max_new");
    if (B == 0 && N > 0) refuse("rows of no requests: starts holds one number");
    const int64_t words = (max_new + 63) / 64;
    const Tensor all = at_.make({N * (2 * words + 1)}, at::kInt);
    const Tensor masks = cut(all, 0, N * words, at::kLong), pos = cut(all, 2 * N * words, N);
    masks.unsafeGetTensorImpl()->set_sizes_contiguous({N, words});
    check(moe_tree_masks(i32(parents), static_cast<int>(N), i32(starts), i32(lens),
                         static_cast<int>(B), static_cast<int>(max_new),
                         static_cast<int64_t*>(masks.data_ptr()), i32(pos), error_word(a[4], dev),
                         at_.stream),
          "moe_tree_masks");
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(masks));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(pos));
    return r;
  });
}

// (tokens, draws, parents, starts, ctx_lens, max_path, err, stream)
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&]() -> PyObject* {
    const Tensor &tokens = tensor(a[0], "tokens"), &draws = tensor(a[1], "draws"),
                 &parents = tensor(a[2], "parents"), &starts = tensor(a[3], "starts"),
                 &ctx = tensor(a[4], "ctx_lens");
    const Place at_(tokens, "tokens", a[7]);
    const int dev = at_.dev;
    const int64_t N = length(tokens, "tokens"), B = requests_of(starts, dev);
    fits(N, "tokens");
    vec(tokens, at::kInt, N, "tokens", dev);
    vec(draws, at::kInt, N, "draws", dev);
    vec(parents, at::kInt, N, "parents", dev);
    vec(ctx, at::kInt, B, "ctx_lens", dev);
    const long long max_path = nodes_of(a[5], "max_path");
    const Tensor all = at_.make({B * (max_path + 3)}, at::kInt);
    const Tensor path = cut(all, 0, B * max_path), accepted = cut(all, B * max_path, B),
                 next = cut(all, B * (max_path + 1), B), lens = cut(all, B * (max_path + 2), B);
    path.unsafeGetTensorImpl()->set_sizes_contiguous({B, max_path});
    check(moe_tree_accept(i32(tokens), i32(draws), i32(parents), static_cast<int>(N), i32(starts),
                          i32(ctx), static_cast<int>(B), static_cast<int>(max_path), i32(path),
                          i32(accepted), i32(next), i32(lens), error_word(a[6], dev), at_.stream),
          "moe_tree_accept");
    PyObject* r = PyTuple_New(4);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(path));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(accepted));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(next));
    PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(lens));
    return r;
  });
}

// (q, k_cache, v_cache, block_table, starts, seq_lens, masks, max_new, scale,
//  window, k_scale, v_scale, out, return_lse, workspace, err, stream)
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 17, [&]() -> PyObject* {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"),
                 &vc = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table"),
                 &starts = tensor(a[4], "starts"), &lens = tensor(a[5], "seq_lens");
    const Place at_(kc, "k_cache", a[16]);
    const int dev = at_.dev;
    const moe_kv_cache_t c = kv_cache(kc, vc, a[10], a[11], dev);
    if (q.dim() != 3) refuse("q must be [N, Hq, head_dim]");
    const int64_t N = q.size(0), hq = q.size(1), dim = c.head_dim, B = requests_of(starts, dev);
    rows3(q, vector_type(c), N, hq, dim, "q", dev);
    if (hq < 1 || c.kv_heads < 1 || hq % c.kv_heads) {
      std::ostringstream o;
      o << "Hq=" << hq << " is not a multiple of kv_heads=" << c.kv_heads;
      refuse(o.str());
    }
    const Table t = block_table(table, B, dev);
    vec(lens, at::kInt, B, "seq_lens", dev);
    if (hq > (1 << 20) || N > INT32_MAX / hq || t.width > INT32_MAX) refuse("sizes must fit 32 bits");
    const long long max_new = nodes_of(a[7], "max_new");
    const int64_t* masks = nullptr;
    if (a[6] != Py_None) {
      const Tensor& m = tensor(a[6], "masks");
      if (matrix(m, at::kLong, N, "masks", dev) != (max_new + 63) / 64)
        refuse("masks must have a word for every 64 of max_new");
      masks = static_cast<const int64_t*>(m.data_ptr());
    }
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(dim)) : number(a[8]);
    const long long window = integer(a[9], "window");
    Tensor out;
    if (a[12] == Py_None) {
      out = at_.make({N, hq, dim}, vector_type(c));
    } else {
      out = tensor(a[12], "out");
      rows3(out, vector_type(c), N, hq, dim, "out", dev);
    }
    const int with_lse = PyObject_IsTrue(a[13]);
    if (with_lse < 0) throw Raised{};
    Tensor lse;
    if (with_lse) lse = at_.make({N, hq}, at::kFloat);
    const size_t need = moe_attn_tree_workspace(c.kv_dtype, c.head_dim);
    c10::DataPtr own;  // returned to the stream's pool when the call has been enqueued
    void* ws;
    size_t bytes = need;
    if (a[14] == Py_None) {
      own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
      ws = own.get();
    } else {
      const Tensor& w = tensor(a[14], "workspace");
      bytes = static_cast<size_t>(length(w, "workspace"));
      ws = vec(w, at::kByte, w.size(0), "workspace", dev);
    }
    check(moe_attn_tree(&c, q.data_ptr(), stride_of(q, 0), stride_of(q, 1), static_cast<int>(N),
                        static_cast<int>(hq), t.p, static_cast<int>(t.width), t.stride, i32(starts),
                        i32(lens), static_cast<int>(B), masks, static_cast<int>(max_new),
                        static_cast<float>(scale), static_cast<int>(window), out.data_ptr(),
                        stride_of(out, 0), stride_of(out, 1),
                        with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws, bytes,
                        error_word(a[15], dev), at_.stream),
          "moe_attn_tree");
    if (a[12] != Py_None) written(out);
    if (!with_lse) return THPVariable_Wrap(out);
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
    return r;
  });
}

// (path, accepted, ctx_lens, block_table, k_cache, v_cache, err, stream)
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&]() -> PyObject* {
    const Tensor &path = tensor(a[0], "path"), &accepted = tensor(a[1], "accepted"),
                 &ctx = tensor(a[2], "ctx_lens"), &table = tensor(a[3], "block_table"),
                 &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache");
    const Place at_(kc, "k_cache", a[7]);
    const int dev = at_.dev;
    const moe_kv_cache_t c = kv_cache(kc, vc, dev);
    const int64_t B = length(accepted, "accepted");
    fits(B, "accepted");
    vec(accepted, at::kInt, B, "accepted", dev);
    vec(ctx, at::kInt, B, "ctx_lens", dev);
    const int64_t P = matrix(path, at::kInt, B, "path", dev);
    const Table t = block_table(table, B, dev);
    fits(t.width, "block_table");
    check(moe_kv_compact(&c, i32(path), static_cast<int>(P), i32(accepted), i32(ctx),
                         static_cast<int>(B), t.p, static_cast<int>(t.width), t.stride,
                         error_word(a[6], dev), at_.stream),
          "moe_kv_compact");
    written(kc);
    written(vc);
    Py_RETURN_NONE;
  });
}

// (src_pages, dst_pages, k_cache, v_cache, tokens, err, stream)
PyObject* kv_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const Tensor &src = tensor(a[0], "src_pages"), &dst = tensor(a[1], "dst_pages"),
                 &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
    const Place at_(kc, "k_cache", a[6]);
    const int dev = at_.dev;
    const moe_kv_cache_t c = kv_cache(kc, vc, dev);
    const int64_t F = length(src, "src_pages");
    fits(F, "src_pages");
    vec(src, at::kInt, F, "src_pages", dev);
    vec(dst, at::kInt, F, "dst_pages", dev);
    check(moe_kv_copy_pages(&c, i32(src), i32(dst),
                            static_cast<int32_t*>(optional_vec(a[4], at::kInt, F, "tokens", dev)),
                            static_cast<int>(F), error_word(a[5], dev), at_.stream),
          "moe_kv_copy_pages");
    written(kc);
    written(vc);
    Py_RETURN_NONE;
  });
}

// (src_rows, dst_rows, ctx_lens, block_table, page_refs, free_pages, n_free,
//  page_size, num_pages, err, stream)
PyObject* kv_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 11, [&]() -> PyObject* {
    const Tensor &src = tensor(a[0], "src_rows"), &dst = tensor(a[1], "dst_rows"),
                 &ctx = tensor(a[2], "ctx_lens"), &table = tensor(a[3], "block_table"),
                 &refs = tensor(a[4], "page_refs"), &free = tensor(a[5], "free_pages"),
                 &left = tensor(a[6], "n_free");
    const Place at_(ctx, "ctx_lens", a[10]);
    const int dev = at_.dev;
    const int64_t F = length(src, "src_rows"), B = length(ctx, "ctx_lens"),
                  cap = length(free, "free_pages");
    vec(src, at::kInt, F, "src_rows", dev);
    vec(dst, at::kInt, F, "dst_rows", dev);
    vec(ctx, at::kInt, B, "ctx_lens", dev);
    vec(free, at::kInt, cap, "free_pages", dev);
    vec(left, at::kInt, 1, "n_free", dev);
    const long long page = integer(a[7], "page_size"), pages = integer(a[8], "num_pages");
    vec(refs, at::kInt, pages, "page_refs", dev);
    const Table t = block_table(table, B, dev);
    if (F > INT32_MAX || B > INT32_MAX || cap > INT32_MAX || t.width > INT32_MAX)
      refuse("sizes must fit 32 bits");
    const Tensor all = at_.make({3 * F}, at::kInt);
    const Tensor from = cut(all, 0, F), to = cut(all, F, F), tokens = cut(all, 2 * F, F);
    check(moe_kv_fork(i32(src), i32(dst), static_cast<int>(F), i32(ctx), static_cast<int>(B), t.p,
                      static_cast<int>(t.width), t.stride, i32(refs), i32(free),
                      static_cast<int>(cap), i32(left), static_cast<int>(pages),
                      static_cast<int>(page), i32(from), i32(to), i32(tokens),
                      error_word(a[9], dev), at_.stream),
          "moe_kv_fork");
    written(ctx);
    written(table);
    written(refs);
    written(left);
    PyObject* r = PyTuple_New(3);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(from));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(to));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(tokens));
    return r;
  });
}

// (keep_lens, seq_lens, block_table, free_pages, n_free, page_size, num_pages,
//  page_refs, err, stream)
PyObject* kv_trim(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&]() -> PyObject* {
    const Tensor &keep = tensor(a[0], "keep_lens"), &lens = tensor(a[1], "seq_lens"),
                 &table = tensor(a[2], "block_table"), &free = tensor(a[3], "free_pages"),
                 &left = tensor(a[4], "n_free");
    const Place at_(keep, "keep_lens", a[9]);
    const int dev = at_.dev;
    const int64_t B = length(keep, "keep_lens"), cap = length(free, "free_pages");
    vec(keep, at::kInt, B, "keep_lens", dev);
    vec(lens, at::kInt, B, "seq_lens", dev);
    vec(free, at::kInt, cap, "free_pages", dev);
    vec(left, at::kInt, 1, "n_free", dev);
    const long long page = integer(a[5], "page_size"), pages = integer(a[6], "num_pages");
    void* const refs = optional_vec(a[7], at::kInt, pages, "page_refs", dev);
    const Table t = block_table(table, B, dev);
    if (B > INT32_MAX || cap > INT32_MAX || t.width > INT32_MAX) refuse("sizes must fit 32 bits");
    check(moe_kv_trim(i32(keep), i32(lens), static_cast<int>(B), t.p, static_cast<int>(t.width),
                      t.stride, i32(free), static_cast<int>(cap), i32(left),
                      static_cast<int32_t*>(refs), static_cast<int>(pages), static_cast<int>(page),
                      error_word(a[8], dev), at_.stream),
          "moe_kv_trim");
    written(table);
    written(free);
    written(left);
    if (refs) written(tensor(a[7], "page_refs"));
    Py_RETURN_NONE;
  });
}

// [n, V] with contiguous rows
void logits_of(const Tensor& x, const char* name) {
  if (x.scalar_type() != at::kFloat && x.scalar_type() != at::kBFloat16)
    refuse(std::string(name) + " must be float32 or bfloat16");
  if (x.dim() != 2 || x.size(1) < 1 || (x.size(1) > 1 && x.stride(1) != 1))
    refuse(std::string(name) + " must be [N, V] with contiguous rows");
}

// (logits, rows, history, history_lens, prompt_lens, repetition, presence,
//  frequency, bias_ids, bias, allowed, tokens, masks, starts, out, err, stream)
PyObject* adjust_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 17, [&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "logits");
    const Place at_(x, "logits", a[16]);
    const int dev = at_.dev;
    logits_of(x, "logits");
    const int64_t N = x.size(0), V = x.size(1);
    if (N > INT32_MAX || V > INT32_MAX) refuse("sizes must fit 32 bits");
    moe_adjust_t s = {};
    s.rows = static_cast<const int32_t*>(optional_vec(a[1], at::kInt, N, "rows", dev));
    // requests: as many as the first tensor that speaks of them has
    int64_t R = -1;
    for (int i = 2; i < 10 && R < 0; ++i)
      if (a[i] != Py_None) {
        const Tensor& t = tensor(a[i], "a request's setting");
        if (t.dim() < 1) refuse("settings must have a row per request");
        R = t.size(0);
      }
    if (R < 0) R = s.rows ? INT32_MAX : N;
    if (!s.rows && R != N) refuse("settings must have a row for each of logits, or rows must be given");
    fits(R, "requests");
    s.requests = static_cast<int32_t>(R);
    if (a[2] != Py_None) {
      const Tensor& h = tensor(a[2], "history");
      on_device(h, "history", dev);
      of_type(h, at::kInt, "history");
      if (h.dim() != 2 || h.size(0) != R || h.size(1) > INT32_MAX ||
          (h.size(1) > 1 && h.stride(1) != 1) || (R > 1 && h.stride(0) < 0))
        refuse("history must be [requests, length] with contiguous rows");
      if (a[3] == Py_None) refuse("history needs history_lens");
      s.history = i32(h);
      s.max_history = static_cast<int32_t>(h.size(1));
      s.history_stride = R > 1 ? h.stride(0) : h.size(1);
    } else {
      for (int i = 3; i < 8; ++i)
        if (a[i] != Py_None)
          refuse("history_lens, prompt_lens and penalties are only used with a history");
      if (a[11] != Py_None) refuse("drafted tokens are only used with a history");
    }
    s.history_lens = static_cast<const int32_t*>(optional_vec(a[3], at::kInt, R, "history_lens", dev));
    s.prompt_lens = static_cast<const int32_t*>(optional_vec(a[4], at::kInt, R, "prompt_lens", dev));
    s.repetition = static_cast<const float*>(optional_vec(a[5], at::kFloat, R, "repetition", dev));
    s.presence = static_cast<const float*>(optional_vec(a[6], at::kFloat, R, "presence", dev));
    s.frequency = static_cast<const float*>(optional_vec(a[7], at::kFloat, R, "frequency", dev));
    if ((a[8] == Py_None) != (a[9] == Py_None)) refuse("bias_ids and bias come together");
    if (a[8] != Py_None) {
      const Tensor &ids = tensor(a[8], "bias_ids"), &bias = tensor(a[9], "bias");
      const int64_t m = matrix(ids, at::kInt, R, "bias_ids", dev);
      if (matrix(bias, at::kFloat, R, "bias", dev) != m)
        refuse("bias must have the shape of bias_ids");
      s.n_bias = static_cast<int32_t>(m);
      s.bias_ids = i32(ids);
      s.bias = static_cast<const float*>(bias.data_ptr());
    }
    if (a[10] != Py_None) {
      const Tensor& w = tensor(a[10], "allowed");
      on_device(w, "allowed", dev);
      of_type(w, at::kInt, "allowed");
      if (w.dim() != 2 || w.size(0) != N || w.size(1) < (V + 31) / 32 ||
          (w.size(1) > 1 && w.stride(1) != 1)) {
        std::ostringstream o;
        o << "allowed must have shape (" << N << ", >= " << (V + 31) / 32
          << ") and contiguous rows, got " << shape_text(w.sizes());
        refuse(o.str());
      }
      s.allowed = i32(w);
      s.allowed_stride = N > 1 ? w.stride(0) : w.size(1);
    }
    if ((a[11] == Py_None) != (a[12] == Py_None) || (a[11] == Py_None) != (a[13] == Py_None))
      refuse("tokens, masks and starts come together");
    if (a[11] != Py_None) {
      const Tensor& m = tensor(a[12], "masks");
      const int64_t words = matrix(m, at::kLong, N, "masks", dev);
      if (words < 1 || words > MOE_TREE_MAX / 64)
        refuse("masks must have a word for every 64 nodes, " + std::to_string(MOE_TREE_MAX / 64) +
               " at most");
      s.mask_words = static_cast<int32_t>(words);
      s.masks = static_cast<const int64_t*>(m.data_ptr());
      s.tokens = static_cast<const int32_t*>(optional_vec(a[11], at::kInt, N, "tokens", dev));
      s.starts = static_cast<const int32_t*>(optional_vec(a[13], at::kInt, R + 1, "starts", dev));
    }
    Tensor out;
    if (a[14] == Py_None) {
      out = at_.make({N, V}, x.scalar_type());
    } else {
      out = tensor(a[14], "out");
      on_device(out, "out", dev);
      logits_of(out, "out");
      if (out.scalar_type() != x.scalar_type() || out.sizes() != x.sizes())
        refuse("out must have logits' type and shape");
    }
    check(moe_adjust_logits(&s, x.data_ptr(),
                            x.scalar_type() == at::kFloat ? MOE_LOGITS_F32 : MOE_LOGITS_BF16,
                            static_cast<int>(N), static_cast<int>(V), N > 1 ? x.stride(0) : V,
                            out.data_ptr(), N > 1 ? out.stride(0) : V, error_word(a[15], dev),
                            at_.stream),
          "moe_adjust_logits");
    if (a[14] == Py_None) return THPVariable_Wrap(out);
    written(out);
    Py_INCREF(a[14]);
    return a[14];
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {
    {"kv_step", fast<kv_step>(), METH_FASTCALL, nullptr},
    {"kv_release", fast<kv_release>(), METH_FASTCALL, nullptr},
    {"kv_append", fast<kv_append>(), METH_FASTCALL, nullptr},
    {"attn_decode", fast<attn_decode>(), METH_FASTCALL, nullptr},
    {"sample_tokens", fast<sample_tokens>(), METH_FASTCALL, nullptr},
    {"tree_masks", fast<tree_masks>(), METH_FASTCALL, nullptr},
    {"tree_accept", fast<tree_accept>(), METH_FASTCALL, nullptr},
    {"attn_tree", fast<attn_tree>(), METH_FASTCALL, nullptr},
    {"kv_compact", fast<kv_compact>(), METH_FASTCALL, nullptr},
    {"kv_copy_pages", fast<kv_copy_pages>(), METH_FASTCALL, nullptr},
    {"kv_fork", fast<kv_fork>(), METH_FASTCALL, nullptr},
    {"kv_trim", fast<kv_trim>(), METH_FASTCALL, nullptr},
    {"adjust_logits", fast<adjust_logits>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "moe_decode_ext", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_decode_ext() { return PyModule_Create(&kModule); }
