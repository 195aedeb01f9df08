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

moe_kv_cache_t kv_cache(const Tensor& k, const Tensor& v, PyObject* k_scale, PyObject* v_scale,
                        int dev) {
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

// n elements of a buffer, from `at` on, as a tensor of its own
Tensor cut(const Tensor& buffer, int64_t at, int64_t n) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()),
                                                      buffer.key_set(), buffer.dtype());
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
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "moe_decode_ext", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_decode_ext() { return PyModule_Create(&kModule); }
