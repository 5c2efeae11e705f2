// Python entry to the paged K/V cache operators: checks the tensors' device,
// type, shape and strides, allocates what the caller did not give, and calls
// the C entry points (whose addresses the package passes to init).  Single-token
// steps are bound by the host, and this takes a third to a half of what the same
// checks and allocations took in Python.
#include <Python.h>

#include <climits>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/smla.h"

namespace {

decltype(&paged_blocks_extend) g_extend;
decltype(&paged_blocks_release) g_release;
decltype(&kv_cache_store_fp8) g_store;
decltype(&paged_attention_fp8) g_attention;
decltype(&paged_attention_fp8_workspace_bytes) g_workspace_bytes;
decltype(&smla_last_error) g_last_error;
PyObject* g_error;

// Thrown once the Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  PyErr_SetString(g_error, text);
  throw Refused();
}

struct Shape {
  int n;
  int64_t d[4];
};

void print_shape(char* to, size_t size, at::IntArrayRef d) {
  size_t at = (size_t)snprintf(to, size, "(");
  for (size_t i = 0; i < d.size() && at < size; ++i)
    at += (size_t)snprintf(to + at, size - at, i ? ", %lld" : "%lld", (long long)d[i]);
  if (at < size) snprintf(to + at, size - at, ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s: must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse("all tensors must be CUDA tensors (there is no CPU path)");
  return t;
}

// The device that all tensors of a call are on.
struct Device {
  int index = -1;
  void same(const at::Tensor& t) {
    const int d = t.get_device();
    if (index < 0) index = d;
    else if (d != index) refuse("all tensors must be on the same device");
  }
};

void check_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type) refuse("%s: dtype %s, expected %s", name, c10::toString(t.scalar_type()), c10::toString(type));
}

void check_shape(const at::Tensor& t, const Shape& shape, const char* name) {
  bool ok = t.dim() == shape.n;
  for (int i = 0; ok && i < shape.n; ++i) ok = t.size(i) == shape.d[i];
  if (ok) return;
  char is[128], want[128];
  print_shape(is, sizeof(is), t.sizes());
  print_shape(want, sizeof(want), at::IntArrayRef(shape.d, (size_t)shape.n));
  refuse("%s: shape %s, expected %s", name, is, want);
}

// A contiguous tensor of this type and shape.
const at::Tensor& arg(PyObject* o, const char* name, at::ScalarType type, const Shape& shape, Device& dev) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, type, name);
  check_shape(t, shape, name);
  if (!t.is_contiguous()) refuse("all tensors must be contiguous");
  dev.same(t);
  return t;
}

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// The same, or null for None.
template <typename T>
T* optional(PyObject* o, const char* name, at::ScalarType type, const Shape& shape, Device& dev) {
  return o == Py_None ? nullptr : data<T>(arg(o, name, type, shape, dev));
}

// [T, heads, D] bf16 rows that may be slices of longer ones; their distance in elements.
int64_t rows(const at::Tensor& t, const char* name, int64_t heads, int64_t D, Device& dev) {
  dev.same(t);
  check_type(t, at::kBFloat16, name);
  check_shape(t, {3, {t.dim() == 3 ? t.size(0) : 0, heads, D}}, name);
  if (t.size(0) > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D)))
    refuse("%s: the heads of a token must be contiguous", name);
  return t.size(0) > 1 ? t.stride(0) : heads * D;
}

int integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < INT_MIN || v > INT_MAX) refuse("%s: %lld is out of range", name, v);
  return (int)v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

int size(int64_t v, const char* name) {
  if (v > INT_MAX) refuse("%s: %lld is out of range", name, (long long)v);
  return (int)v;
}

struct Table {
  int R, MB;
};
Table table(const at::Tensor& t) {
  if (t.dim() != 2) {
    char is[128];
    print_shape(is, sizeof(is), t.sizes());
    refuse("block_table: shape %s, expected (R, MB)", is);
  }
  return {size(t.size(0), "R"), size(t.size(1), "MB")};
}

struct Cache {
  int NB, HK, D;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
};
Cache cache(PyObject* const* a, Device& dev) {
  const at::Tensor& k = tensor(a[0], "k_cache");
  if (k.dim() != 4 || k.size(2) != 64) {
    char is[128];
    print_shape(is, sizeof(is), k.sizes());
    refuse("k_cache: shape %s, expected (NB, HK, 64, D)", is);
  }
  Cache c;
  c.NB = size(k.size(0), "NB");
  c.HK = size(k.size(1), "HK");
  c.D = size(k.size(3), "D");
  const Shape codes{4, {c.NB, c.HK, 64, c.D}}, scales{2, {c.NB, c.HK}};
  c.k = data<uint8_t>(arg(a[0], "k_cache", at::kByte, codes, dev));
  c.v = data<uint8_t>(arg(a[1], "v_cache", at::kByte, codes, dev));
  c.k_scale = data<float>(arg(a[2], "k_scale", at::kFloat, scales, dev));
  c.v_scale = data<float>(arg(a[3], "v_scale", at::kFloat, scales, dev));
  return c;
}

at::Tensor made(at::IntArrayRef shape, at::ScalarType type, const Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev.index));
}

void check(int rc, const char* what) {
  if (rc != SMLA_OK) refuse("%s failed with status %d: %s", what, rc, g_last_error());
}

// Runs `body` (which returns a new reference), turning what it throws into a Python error.
template <typename F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Refused();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw Refused();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void expect_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
    throw Refused();
  }
}

// (context_lens, query_lens, block_table, free_blocks, free_count, num_tokens, num_blocks, out or None)
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 8);
    Device dev;
    const at::Tensor& bt = tensor(a[2], "block_table");
    const Table tab = table(bt);
    const at::Tensor& fb = tensor(a[3], "free_blocks");
    const int R = tab.R, F = size(fb.numel(), "F"), T = integer(a[5], "num_tokens"), NB = integer(a[6], "num_blocks");
    const auto i32 = at::kInt;
    const int32_t* ctx = data<int32_t>(arg(a[0], "context_lens", i32, {1, {R}}, dev));
    const int32_t* len = data<int32_t>(arg(a[1], "query_lens", i32, {1, {R}}, dev));
    arg(a[2], "block_table", i32, {2, {R, tab.MB}}, dev);
    arg(a[3], "free_blocks", i32, {1, {F}}, dev);
    const int32_t* count = data<int32_t>(arg(a[4], "free_count", i32, {1, {1}}, dev));
    if (T < 0) refuse("num_tokens: %d must not be negative", T);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    static const char* const names[7] = {"query_start", "seq_lens", "req_id_per_token", "positions", "slot_mapping",
                                         "free_count", "missing"};
    const int64_t sizes[7] = {R + 1, R, T, T, T, 1, 1};
    at::Tensor out[7];
    if (a[7] == Py_None) {
      for (int i = 0; i < 7; ++i) out[i] = made({sizes[i]}, i == 4 ? at::kLong : i32, dev);
    } else {
      if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 7) refuse("out: must be a PagedBatch");
      for (int i = 0; i < 7; ++i)
        out[i] = arg(PyTuple_GET_ITEM(a[7], i), names[i], i == 4 ? at::kLong : i32, {1, {sizes[i]}}, dev);
    }
    check(g_extend(ctx, len, data<int32_t>(bt), data<int32_t>(fb), count, data<int32_t>(out[0]), data<int32_t>(out[1]),
                   data<int32_t>(out[2]), data<int32_t>(out[3]), data<int64_t>(out[4]), data<int32_t>(out[5]),
                   data<int32_t>(out[6]), R, tab.MB, NB, F, T, c10::cuda::getCurrentCUDAStream(dev.index).stream()),
          "paged_blocks_extend");
    if (a[7] != Py_None) {
      Py_INCREF(a[7]);
      return a[7];
    }
    return pack({out[0], out[1], out[2], out[3], out[4], out[5], out[6]});
  });
}

// (release, seq_lens, block_table, free_blocks, free_count, num_blocks, context_lens or None, free_count_out or None)
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 8);
    Device dev;
    const at::Tensor& gone = tensor(a[0], "release");
    const at::Tensor& bt = tensor(a[2], "block_table");
    const Table tab = table(bt);
    const at::Tensor& fb = tensor(a[3], "free_blocks");
    const int R = tab.R, F = size(fb.numel(), "F"), NB = integer(a[5], "num_blocks");
    if (gone.scalar_type() != at::kBool && gone.scalar_type() != at::kByte)
      refuse("release: dtype %s, expected bool or uint8", c10::toString(gone.scalar_type()));
    arg(a[0], "release", gone.scalar_type(), {1, {R}}, dev);
    const int32_t* lens = data<int32_t>(arg(a[1], "seq_lens", at::kInt, {1, {R}}, dev));
    arg(a[2], "block_table", at::kInt, {2, {R, tab.MB}}, dev);
    arg(a[3], "free_blocks", at::kInt, {1, {F}}, dev);
    const int32_t* count = data<int32_t>(arg(a[4], "free_count", at::kInt, {1, {1}}, dev));
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    const at::Tensor ctx =
        a[6] == Py_None ? made({R}, at::kInt, dev) : arg(a[6], "context_lens", at::kInt, {1, {R}}, dev);
    const at::Tensor left =
        a[7] == Py_None ? made({1}, at::kInt, dev) : arg(a[7], "free_count_out", at::kInt, {1, {1}}, dev);
    check(g_release(data<uint8_t>(gone), lens, data<int32_t>(bt), data<int32_t>(fb), count, data<int32_t>(ctx),
                    data<int32_t>(left), R, tab.MB, NB, F, c10::cuda::getCurrentCUDAStream(dev.index).stream()),
          "paged_blocks_release");
    return pack({ctx, left});
  });
}

// (k, v, query_start, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale)
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 9);
    Device dev;
    const at::Tensor& bt = tensor(a[4], "block_table");
    const Table tab = table(bt);
    const int32_t* start = data<int32_t>(arg(a[2], "query_start", at::kInt, {1, {tab.R + 1}}, dev));
    const int32_t* lens = data<int32_t>(arg(a[3], "seq_lens", at::kInt, {1, {tab.R}}, dev));
    arg(a[4], "block_table", at::kInt, {2, {tab.R, tab.MB}}, dev);
    const Cache c = cache(a + 5, dev);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t k_stride = rows(k, "k", c.HK, c.D, dev), v_stride = rows(v, "v", c.HK, c.D, dev);
    const int T = size(k.size(0), "T");
    if (v.size(0) != T) refuse("k has %d tokens, v %lld", T, (long long)v.size(0));
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    check(g_store(k.data_ptr(), k_stride, v.data_ptr(), v_stride, start, lens, data<int32_t>(bt), c.k, c.v, c.k_scale,
                  c.v_scale, T, c.HK, c.D, tab.R, tab.MB, c.NB, c10::cuda::getCurrentCUDAStream(dev.index).stream()),
          "kv_cache_store_fp8");
    Py_RETURN_NONE;
  });
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start, sm_scale, max_query_len or None,
//  window, softcap, alibi_slopes, prefix_lens, doc_start, out, lse, workspace: each or None)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 18);
    Device dev;
    const at::Tensor& bt = tensor(a[5], "block_table");
    const Table tab = table(bt);
    const Cache c = cache(a + 1, dev);
    arg(a[5], "block_table", at::kInt, {2, {tab.R, tab.MB}}, dev);
    const int32_t* lens = data<int32_t>(arg(a[6], "seq_lens", at::kInt, {1, {tab.R}}, dev));
    const int32_t* start = data<int32_t>(arg(a[7], "query_start", at::kInt, {1, {tab.R + 1}}, dev));
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 3) refuse("q: must be [T, H, D]");
    const int T = size(q.size(0), "T"), H = size(q.size(1), "H");
    const int64_t stride = rows(q, "q", H, c.D, dev);
    const int longest = a[9] == Py_None ? std::max(1, T - tab.R + 1) : integer(a[9], "max_query_len");
    const float* slopes = optional<float>(a[12], "alibi_slopes", at::kFloat, {1, {H}}, dev);
    const int32_t* prefix = optional<int32_t>(a[13], "prefix_lens", at::kInt, {1, {tab.R}}, dev);
    const int32_t* doc = optional<int32_t>(a[14], "doc_start", at::kInt, {1, {T}}, dev);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    const at::Tensor out =
        a[15] == Py_None ? made({T, H, c.D}, at::kBFloat16, dev) : arg(a[15], "out", at::kBFloat16, {3, {T, H, c.D}}, dev);
    const at::Tensor lse =
        a[16] == Py_None ? made({T, H}, at::kFloat, dev) : arg(a[16], "lse", at::kFloat, {2, {T, H}}, dev);
    at::Tensor ws;
    if (a[17] == Py_None) {
      ws = made({(int64_t)g_workspace_bytes(T, H, c.HK, c.D, tab.R, longest)}, at::kByte, dev);
    } else {
      ws = tensor(a[17], "workspace");
      if (!ws.is_contiguous()) refuse("all tensors must be contiguous");
      dev.same(ws);
      if (ws.numel() == 0) refuse("workspace: must not be empty");  // (its address, null, would ask for the library's)
    }
    check(g_attention(q.data_ptr(), stride, c.k, c.v, c.k_scale, c.v_scale, data<int32_t>(bt), lens, start, number(a[8]),
                      longest, integer(a[10], "window"), number(a[11]), slopes, prefix, doc, out.data_ptr(),
                      data<float>(lse), T, H, c.HK, c.D, tab.R, tab.MB, c.NB, ws.data_ptr(), (size_t)ws.nbytes(),
                      c10::cuda::getCurrentCUDAStream(dev.index).stream()),
          "paged_attention_fp8");
    return pack({out, lse});
  });
}

// (error class, addresses of the entry points)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "init: 7 arguments expected");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "init: null address");
      return nullptr;
    }
  }
  Py_INCREF(a[0]);
  g_error = a[0];
  g_extend = reinterpret_cast<decltype(g_extend)>(p[0]);
  g_release = reinterpret_cast<decltype(g_release)>(p[1]);
  g_store = reinterpret_cast<decltype(g_store)>(p[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[3]);
  g_workspace_bytes = reinterpret_cast<decltype(g_workspace_bytes)>(p[4]);
  g_last_error = reinterpret_cast<decltype(g_last_error)>(p[5]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {{"init", FAST(init), METH_FASTCALL, nullptr},
                          {"extend", FAST(extend), METH_FASTCALL, nullptr},
                          {"release", FAST(release), METH_FASTCALL, nullptr},
                          {"store", FAST(store), METH_FASTCALL, nullptr},
                          {"attention", FAST(attention), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
