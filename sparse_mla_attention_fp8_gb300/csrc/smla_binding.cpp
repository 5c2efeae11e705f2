// Python entry to the paged K/V cache and the MXFP8 operators: checks the tensors' device,
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
decltype(&mxfp8_quantize) g_quantize;
decltype(&rms_norm_mxfp8) g_norm;
decltype(&linear_mxfp8) g_linear;
decltype(&moe_route) g_route;
decltype(&moe_mxfp8) g_moe;
decltype(&moe_mxfp8_workspace_bytes) g_moe_workspace_bytes;
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

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v == 1;
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

// ---- MXFP8 operators

// A matrix [rows, K] whose rows may be slices of longer ones; their distance in elements.
struct Matrix {
  const at::Tensor* t;
  int rows, K;
  int64_t stride;
};
Matrix matrix(PyObject* o, const char* name, Device& dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2) {
    char is[128];
    print_shape(is, sizeof(is), t.sizes());
    refuse("%s: shape %s, expected (rows, K)", name, is);
  }
  dev.same(t);
  const int rows = size(t.size(0), name), K = size(t.size(1), name);
  if (rows > 0 && K > 1 && t.stride(1) != 1) refuse("%s: the values of a row must be contiguous", name);
  return {&t, rows, K, rows > 1 ? t.stride(0) : (K + 15) / 16 * 16};
}
Matrix matrix_of(PyObject* o, const char* name, at::ScalarType type, int rows, int K, Device& dev) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, type, name);
  check_shape(t, {2, {rows, K}}, name);
  return matrix(o, name, dev);
}

// Codes as bytes or as e4m3 values, scales as bytes or as e8m0 values.
void check_code_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat8_e4m3fn)
    refuse("%s: dtype %s, expected uint8 or float8_e4m3fn", name, c10::toString(t.scalar_type()));
}
Matrix code_rows(PyObject* o, const char* name, Device& dev) {
  check_code_type(tensor(o, name), name);
  return matrix(o, name, dev);
}
uint8_t* codes(PyObject* o, const char* name, const Shape& shape, Device& dev) {
  const at::Tensor& t = tensor(o, name);
  check_code_type(t, name);
  return static_cast<uint8_t*>(arg(o, name, t.scalar_type(), shape, dev).data_ptr());
}
struct Scales {
  uint8_t* p;
  int64_t stride;
};
// [rows, K / 32], or [E, rows / E, K / 32] with all rows one distance apart.
Scales scales(PyObject* o, const char* name, int64_t E, int64_t rows, int64_t K, Device& dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat8_e8m0fnu)
    refuse("%s: dtype %s, expected uint8 or float8_e8m0fnu", name, c10::toString(t.scalar_type()));
  const int64_t n = K / 32;
  check_shape(t, E ? Shape{3, {E, rows, n}} : Shape{2, {rows, n}}, name);
  dev.same(t);
  const int d = E ? 1 : 0;
  const int64_t padded = (n + 3) / 4 * 4, stride = rows > 1 ? t.stride(d) : E > 1 ? t.stride(0) : padded;
  if (rows > 0 && n > 1 && t.stride(d + 1) != 1) refuse("%s: the scales of a row must be contiguous", name);
  if (E > 1 && rows > 1 && t.stride(0) != rows * stride) refuse("%s: all rows must be one distance apart", name);
  return {static_cast<uint8_t*>(t.data_ptr()), stride};
}
// 16 bytes, not 4: rows on 16-byte boundaries can be copied by TMA (the linear product's kernel for many tokens).
int64_t made_scale_stride(int64_t K) { return (K / 32 + 15) / 16 * 16; }
// uint8 [rows, cols] of `from`'s memory, from byte `offset` on, rows `stride` bytes apart.
at::Tensor bytes_of(const at::Tensor& from, int64_t offset, int64_t rows, int64_t cols, int64_t stride) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(from.storage()), from.key_set(), from.dtype());
  const int64_t sizes[2] = {rows, cols}, strides[2] = {stride, 1};
  t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides, offset);
  return t;
}
// Where quantized results go: what the caller gave, or new tensors.
struct Quantized {
  at::Tensor codes, scales;
  uint8_t *c, *s;
  int64_t stride;
};
Quantized quantized(PyObject* c, PyObject* s, const char* cname, const char* sname, int rows, int K, Device& dev) {
  if (K <= 0 || K % 32 != 0) refuse("%d values a row: must be a positive multiple of 32", K);
  Quantized q;
  const int64_t stride = made_scale_stride(K);
  if (c == Py_None && s == Py_None) {
    // one allocation for both: an allocation is a fifth of the time that the host takes for a small call
    const int64_t behind = ((int64_t)rows * K + 255) / 256 * 256;
    const at::Tensor both = made({behind + rows * stride}, at::kByte, dev);
    q.codes = bytes_of(both, 0, rows, K, K);
    q.scales = bytes_of(both, behind, rows, K / 32, stride);
    q.c = data<uint8_t>(both);
    q.s = q.c + behind;
    q.stride = stride;
    return q;
  }
  if (c == Py_None) {
    q.codes = made({rows, K}, at::kByte, dev);
    q.c = data<uint8_t>(q.codes);
  } else {
    q.c = codes(c, cname, {2, {rows, K}}, dev);
    q.codes = THPVariable_Unpack(c);
  }
  if (s == Py_None) {
    q.scales = bytes_of(made({rows * stride}, at::kByte, dev), 0, rows, K / 32, stride);
    q.s = data<uint8_t>(q.scales);
    q.stride = stride;
  } else {
    const Scales given = scales(s, sname, 0, rows, K, dev);
    q.scales = THPVariable_Unpack(s);
    q.s = given.p;
    q.stride = given.stride;
  }
  return q;
}
// bf16 or float32
int float_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SMLA_BF16;
  if (t.scalar_type() == at::kFloat) return SMLA_F32;
  refuse("%s: dtype %s, expected bfloat16 or float32", name, c10::toString(t.scalar_type()));
}
void* stream_of(const Device& dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream(); }

// (x, codes or None, scales or None)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 3);
    Device dev;
    const Matrix x = matrix(a[0], "x", dev);
    const int type = float_type(*x.t, "x");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    const Quantized q = quantized(a[1], a[2], "codes", "scales", x.rows, x.K, dev);
    check(g_quantize(x.t->data_ptr(), type, x.stride, q.c, q.s, q.stride, x.rows, x.K, stream_of(dev)), "mxfp8_quantize");
    return pack({q.codes, q.scales});
  });
}

// What the caller gave or, for True, a new bf16 [T, K]; undefined for None and False.
at::Tensor wanted(PyObject* o, const char* name, int T, int K, Device& dev) {
  if (o == Py_None || o == Py_False) return {};
  return o == Py_True ? made({T, K}, at::kBFloat16, dev) : arg(o, name, at::kBFloat16, {2, {T, K}}, dev);
}
PyObject* or_none(const at::Tensor& t) {
  if (t.defined()) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) throw Refused();
    return o;
  }
  Py_RETURN_NONE;
}

// (x, weight or None, eps, residual or None, normed, quantized, residual_out or None, codes or None, scales or None)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 9);
    Device dev;
    const Matrix x = matrix(a[0], "x", dev);
    check_type(*x.t, at::kBFloat16, "x");
    const int T = x.rows, K = x.K;
    const void* weight = nullptr;
    int type = SMLA_BF16;
    if (a[1] != Py_None) {
      const at::Tensor& w = tensor(a[1], "weight");
      type = float_type(w, "weight");
      weight = arg(a[1], "weight", w.scalar_type(), {1, {K}}, dev).data_ptr();
    }
    Matrix res{};
    if (a[3] != Py_None) res = matrix_of(a[3], "residual", at::kBFloat16, T, K, dev);
    const bool codes_too = truth(a[5]);
    if (!codes_too && (a[7] != Py_None || a[8] != Py_None)) refuse("codes and scales: given, but not asked for (quantized)");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    Quantized q{};
    if (codes_too) q = quantized(a[7], a[8], "codes", "scales", T, K, dev);
    const at::Tensor normed = wanted(a[4], "normed", T, K, dev);
    const at::Tensor h = wanted(a[6] == Py_None && res.t ? Py_True : a[6], "residual_out", T, K, dev);
    check(g_norm(x.t->data_ptr(), x.stride, res.t ? res.t->data_ptr() : nullptr, res.stride, weight, type, number(a[2]), q.c,
                 q.s, q.stride, normed.defined() ? normed.data_ptr() : nullptr, h.defined() ? h.data_ptr() : nullptr, T, K,
                 stream_of(dev)),
          "rms_norm_mxfp8");
    PyObject* r = PyTuple_New(4);
    if (!r) throw Refused();
    const at::Tensor* all[4] = {&q.codes, &q.scales, &normed, &h};
    for (int i = 0; i < 4; ++i) {
      try {
        PyTuple_SET_ITEM(r, i, or_none(*all[i]));
      } catch (...) {
        Py_DECREF(r);
        throw;
      }
    }
    return r;
  });
}

// (x, x_scale, weight, weight_scale, bias or None, activation, residual or None, quantized, out or None, out_scale or None)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 10);
    Device dev;
    const Matrix x = code_rows(a[0], "x", dev);
    const int T = x.rows, K = x.K, act = integer(a[5], "activation");
    const Scales xs = scales(a[1], "x_scale", 0, T, K, dev);
    const Matrix w = code_rows(a[2], "weight", dev);
    if (w.K != K) refuse("weight: shape (%d, %d), expected (N, %d)", w.rows, w.K, K);
    if (!w.t->is_contiguous()) refuse("all tensors must be contiguous");
    if (act == SMLA_ACT_SWIGLU && w.rows % 2 != 0) refuse("weight: %d rows, which must be even for swiglu", w.rows);
    const int N = act == SMLA_ACT_SWIGLU ? w.rows / 2 : w.rows;
    const Scales ws = scales(a[3], "weight_scale", 0, w.rows, K, dev);
    const void* bias = nullptr;
    int type = SMLA_BF16;
    if (a[4] != Py_None) {
      const at::Tensor& b = tensor(a[4], "bias");
      type = float_type(b, "bias");
      bias = arg(a[4], "bias", b.scalar_type(), {1, {w.rows}}, dev).data_ptr();
    }
    Matrix res{};
    if (a[6] != Py_None) {
      res = matrix_of(a[6], "residual", at::kBFloat16, T, N, dev);
      if (T <= 1) res.stride = N;
    }
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    Quantized q{};
    at::Tensor out;
    const bool coded = truth(a[7]);
    if (!coded && a[9] != Py_None) refuse("out_scale: given, but not asked for (quantized)");
    if (coded)
      q = quantized(a[8], a[9], "out", "out_scale", T, N, dev);
    else
      out = a[8] == Py_None ? made({T, N}, at::kBFloat16, dev) : arg(a[8], "out", at::kBFloat16, {2, {T, N}}, dev);
    check(g_linear(data<uint8_t>(*x.t), x.stride, xs.p, xs.stride, data<uint8_t>(*w.t), ws.p, ws.stride, bias, type, act,
                   res.t ? res.t->data_ptr() : nullptr, res.stride, coded ? nullptr : out.data_ptr(), q.c, q.s, q.stride, T,
                   N, K, stream_of(dev)),
          "linear_mxfp8");
    return coded ? pack({q.codes, q.scales}) : or_none(out);
  });
}

// (logits, topk, scoring, bias or None, renormalize, scale, num_groups, topk_groups, ids or None, weights or None)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 10);
    Device dev;
    const at::Tensor& x = tensor(a[0], "logits");
    if (x.dim() != 2) refuse("logits: must be [T, E]");
    const int T = size(x.size(0), "T"), E = size(x.size(1), "E"), topk = integer(a[1], "topk");
    const int type = float_type(x, "logits");
    arg(a[0], "logits", x.scalar_type(), {2, {T, E}}, dev);
    const float* bias = optional<float>(a[3], "bias", at::kFloat, {1, {E}}, dev);
    if (topk <= 0) refuse("topk: %d must be positive", topk);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    const at::Tensor ids = a[8] == Py_None ? made({T, topk}, at::kInt, dev) : arg(a[8], "ids", at::kInt, {2, {T, topk}}, dev);
    const at::Tensor w =
        a[9] == Py_None ? made({T, topk}, at::kFloat, dev) : arg(a[9], "weights", at::kFloat, {2, {T, topk}}, dev);
    check(g_route(x.data_ptr(), type, bias, integer(a[2], "scoring"), truth(a[4]), number(a[5]),
                  integer(a[6], "num_groups"), integer(a[7], "topk_groups"), data<int32_t>(ids), data<float>(w), T, E, topk,
                  stream_of(dev)),
          "moe_route");
    return pack({ids, w});
  });
}

// (x, x_scale, topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, residual, out, workspace: each or None)
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect_args(n, 11);
    Device dev;
    const Matrix x = code_rows(a[0], "x", dev);
    const int T = x.rows, K = x.K;
    const Scales xs = scales(a[1], "x_scale", 0, T, K, dev);
    const at::Tensor &ids = tensor(a[2], "topk_ids"), &w13 = tensor(a[4], "w13");
    if (ids.dim() != 2) refuse("topk_ids: must be [T, topk]");
    if (w13.dim() != 3 || w13.size(1) % 2 != 0) refuse("w13: must be [E, 2 F, K]");
    const int topk = size(ids.size(1), "topk"), E = size(w13.size(0), "E"), F = size(w13.size(1) / 2, "F");
    arg(a[2], "topk_ids", at::kInt, {2, {T, topk}}, dev);
    const float* weights = data<float>(arg(a[3], "topk_weights", at::kFloat, {2, {T, topk}}, dev));
    const uint8_t* up = codes(a[4], "w13", {3, {E, 2 * (int64_t)F, K}}, dev);
    const Scales ups = scales(a[5], "w13_scale", E, 2 * (int64_t)F, K, dev);
    const uint8_t* down = codes(a[6], "w2", {3, {E, K, F}}, dev);
    const Scales downs = scales(a[7], "w2_scale", E, K, F, dev);
    Matrix res{};
    if (a[8] != Py_None) res = matrix_of(a[8], "residual", at::kBFloat16, T, K, dev);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    const at::Tensor out = a[9] == Py_None ? made({T, K}, at::kBFloat16, dev) : arg(a[9], "out", at::kBFloat16, {2, {T, K}}, dev);
    at::Tensor ws;
    if (a[10] == Py_None) {
      ws = made({(int64_t)g_moe_workspace_bytes(T, E, topk, F)}, at::kByte, dev);
    } else {
      ws = tensor(a[10], "workspace");
      if (!ws.is_contiguous()) refuse("all tensors must be contiguous");
      dev.same(ws);
      if (ws.numel() == 0) refuse("workspace: must not be empty");  // (its address, null, would ask for the library's)
    }
    check(g_moe(data<uint8_t>(*x.t), x.stride, xs.p, xs.stride, data<int32_t>(ids), weights, up, ups.p, ups.stride, down,
                downs.p, downs.stride, res.t ? res.t->data_ptr() : nullptr, res.stride, out.data_ptr(), T, E, topk, K, F,
                ws.data_ptr(), (size_t)ws.nbytes(), stream_of(dev)),
          "moe_mxfp8");
    return or_none(out);
  });
}

// (error class, addresses of the entry points)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kEntries = 12;
  if (n != 1 + kEntries) {
    PyErr_Format(PyExc_TypeError, "init: %d arguments expected", 1 + kEntries);
    return nullptr;
  }
  void* p[kEntries];
  for (int i = 0; i < kEntries; ++i) {
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
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[6]);
  g_norm = reinterpret_cast<decltype(g_norm)>(p[7]);
  g_linear = reinterpret_cast<decltype(g_linear)>(p[8]);
  g_route = reinterpret_cast<decltype(g_route)>(p[9]);
  g_moe = reinterpret_cast<decltype(g_moe)>(p[10]);
  g_moe_workspace_bytes = reinterpret_cast<decltype(g_moe_workspace_bytes)>(p[11]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {{"init", FAST(init), METH_FASTCALL, nullptr},
                          {"extend", FAST(extend), METH_FASTCALL, nullptr},
                          {"release", FAST(release), METH_FASTCALL, nullptr},
                          {"store", FAST(store), METH_FASTCALL, nullptr},
                          {"attention", FAST(attention), METH_FASTCALL, nullptr},
                          {"quantize", FAST(quantize), METH_FASTCALL, nullptr},
                          {"norm", FAST(norm), METH_FASTCALL, nullptr},
                          {"linear", FAST(linear), METH_FASTCALL, nullptr},
                          {"route", FAST(route), METH_FASTCALL, nullptr},
                          {"moe", FAST(moe), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
