// Python entry points of the rotary, page and 8-bit cache calls: tensors checked and handed to
// the C ABI (include/lla.h) on their device's current stream.
//
// A decode step makes these calls for every layer and loop, and between launches of 4 us the
// time to check a dozen tensors counts: attribute by attribute in Python it is 5 to 10 us a
// call, here under 1.  The functions take every argument by position; __init__.py holds their
// signatures and documentation.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "lla.h"

namespace {

using at::ScalarType;

PyObject* g_error = nullptr;      // LLAError
PyObject* g_names[13];            // attributes of Cfg, then of Q8Cache

[[noreturn]] void raise_set() {   // the Python error that is set
  python_error e;
  e.persist();
  throw e;
}

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  raise_set();
}

void check(int code) {
  if (code == LLA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", code, lla_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  raise_set();
}

const char* type_name(ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kChar: return "torch.int8";
    default: return "torch.uint8";
  }
}

std::string shape_text(at::IntArrayRef s) {
  std::string out = "(";
  for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
  return out + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// The tensor whose device the call runs on.
const at::Tensor& leading(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return t;
}

void check_kind(const at::Tensor& t, ScalarType type, c10::Device dev, const char* name) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, "%s must be %s", name, type_name(type));
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.device() != dev)
    fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(),
                            dev.str().c_str());
}

void check_shape(const at::Tensor& t, at::IntArrayRef shape, const char* name) {
  if (t.sizes() != shape)
    fail(PyExc_ValueError, "%s has shape %s, expected %s", name, shape_text(t.sizes()).c_str(),
                            shape_text(shape).c_str());
}

// Address of a contiguous tensor of this type and device.
template <typename T>
T* dense(PyObject* o, ScalarType type, c10::Device dev, const char* name) {
  const at::Tensor& t = tensor(o, name);
  check_kind(t, type, dev, name);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* dense(PyObject* o, ScalarType type, c10::Device dev, const char* name, at::IntArrayRef shape) {
  T* p = dense<T>(o, type, dev, name);
  check_shape(THPVariable_Unpack(o), shape, name);
  return p;
}
int32_t* ints(PyObject* o, c10::Device dev, const char* name, at::IntArrayRef shape) {
  return dense<int32_t>(o, at::kInt, dev, name, shape);
}
int32_t* status_of(PyObject* o, c10::Device dev) {
  if (o == Py_None) return nullptr;
  int32_t* p = dense<int32_t>(o, at::kInt, dev, "status");
  if (THPVariable_Unpack(o).numel() < 1) fail(PyExc_ValueError, "status is empty");
  return p;
}

struct Rows {
  void* p;
  int64_t stride;
};
// Rows [n, heads, d] whose heads are contiguous; tokens may be strided.
Rows rows(PyObject* o, ScalarType type, c10::Device dev, const char* name, at::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name);
  check_kind(t, type, dev, name);
  check_shape(t, shape, name);
  if (t.numel() && !(t.stride(2) == 1 && (shape[1] == 1 || t.stride(1) == shape[2])))
    fail(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
  return {t.data_ptr(), shape[0] > 1 ? t.stride(0) : shape[1] * shape[2]};
}

int row_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return LLA_F32;
  if (t.scalar_type() == at::kBFloat16) return LLA_BF16;
  fail(PyExc_TypeError, "%s must be a float32 or bfloat16 tensor", name);
}

int layout_of(PyObject* o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return LLA_ROPE_HALF;
    if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) return LLA_ROPE_INTERLEAVED;
  }
  fail(PyExc_ValueError, "layout must be 'half' or 'interleaved'");
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) raise_set();
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) fail(PyExc_ValueError, "%s is out of range", name);
  return (int32_t)v;
}

struct Held {                     // a new reference
  PyObject* o;
  explicit Held(PyObject* owned) : o(owned) {
    if (!o) raise_set();
  }
  ~Held() { Py_DECREF(o); }
  Held(const Held&) = delete;
  Held& operator=(const Held&) = delete;
};

lla_cfg config(PyObject* o) {
  static const char* names[] = {"T", "H", "d_head", "r_k", "r_v", "mode", "d_rope"};
  int32_t v[7];
  for (int i = 0; i < 7; ++i) {
    Held a(PyObject_GetAttr(o, g_names[i]));
    v[i] = integer32(a.o, names[i]);
  }
  float f[2];
  for (int i = 0; i < 2; ++i) {
    Held a(PyObject_GetAttr(o, g_names[7 + i]));
    f[i] = (float)PyFloat_AsDouble(a.o);
    if (PyErr_Occurred()) raise_set();
  }
  return {v[0], v[1], v[2], v[3], v[4], v[5], f[0], f[1], v[6]};
}

struct Table {
  float* p = nullptr;
  int32_t positions = 0;
};
// A rope table of the configuration's rotary dims, or None.
Table table_of(PyObject* o, const lla_cfg& c, c10::Device dev) {
  Table t;
  if (o == Py_None) return t;
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 3)
    fail(PyExc_ValueError, "rope must be a table from rope_table, or None");
  const int64_t n = THPVariable_Unpack(o).size(0);
  if (n > INT32_MAX) fail(PyExc_ValueError, "rope has too many positions");
  t.p = dense<float>(o, at::kFloat, dev, "rope", {n, (c.d_rope ? c.d_rope : c.d_head) / 2, 2});
  t.positions = (int32_t)n;
  return t;
}

int32_t small(int64_t n, const char* name) {
  if (n > INT32_MAX) fail(PyExc_ValueError, "%s is too large", name);
  return (int32_t)n;
}

// The cache as the C ABI has it; every array of this configuration and device.
lla_q8_cache cache_of(PyObject* o, const lla_cfg& cfg, c10::Device dev) {
  lla_q8_cache c{};
  Held k(PyObject_GetAttr(o, g_names[9])), v(PyObject_GetAttr(o, g_names[10]));
  Held ks(PyObject_GetAttr(o, g_names[11])), vs(PyObject_GetAttr(o, g_names[12]));
  const at::Tensor& t = tensor(k.o, "cache.k");
  if (t.dim() != 4)
    fail(PyExc_ValueError, "cache.k has shape %s, expected (pages, heads, page, d)",
                            shape_text(t.sizes()).c_str());
  c.n_pages = small(t.size(0), "cache");
  c.page = small(t.size(2), "cache");
  const int64_t shape[] = {t.size(0), cfg.H, t.size(2), cfg.d_head};
  c.k = dense<int8_t>(k.o, at::kChar, dev, "cache.k", shape);
  c.v = dense<int8_t>(v.o, at::kChar, dev, "cache.v", shape);
  c.k_scale = dense<float>(ks.o, at::kFloat, dev, "cache.k_scale", {shape[0], shape[1]});
  c.v_scale = dense<float>(vs.o, at::kFloat, dev, "cache.v_scale", {shape[0], shape[1]});
  return c;
}

struct Pages {
  int32_t* p;
  int32_t B, max_pages;
};
Pages pages_of(PyObject* o, c10::Device dev) {
  const at::Tensor& t = tensor(o, "block_table");
  if (t.dim() != 2) fail(PyExc_ValueError, "block_table must be [B, max_pages]");
  return {dense<int32_t>(o, at::kInt, dev, "block_table"), small(t.size(0), "block_table"),
          small(t.size(1), "block_table")};
}

// An output: the tensor that was given, or a new one for None.
struct Out {
  PyObject* o;
  explicit Out(PyObject* given) : o(given) { Py_INCREF(o); }
  explicit Out(at::Tensor&& made) : o(THPVariable_Wrap(std::move(made))) {
    if (!o) raise_set();
  }
  ~Out() { Py_XDECREF(o); }
  Out(const Out&) = delete;
  Out& operator=(const Out&) = delete;
  PyObject* release() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};
at::Tensor make(at::IntArrayRef shape, ScalarType type, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "expected %d arguments", (int)want);
}

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// (cfg, rope, positions, x, layout, inverse, out, status) -> out
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const lla_cfg cfg = config(a[0]);
  const at::Tensor& x = leading(a[3], "x");
  const int kind = row_type(x, "x");
  const ScalarType type = x.scalar_type();
  const c10::Device dev = x.device();
  if (x.dim() != 3 || x.size(2) != cfg.d_head)
    fail(PyExc_ValueError, "x has shape %s, expected (tokens, heads, %d)",
                            shape_text(x.sizes()).c_str(), cfg.d_head);
  if (a[1] == Py_None) fail(PyExc_ValueError, "rope must be a table from rope_table");
  const c10::cuda::CUDAGuard guard(dev);
  const Table table = table_of(a[1], cfg, dev);
  const int64_t tokens = x.size(0), shape[] = {tokens, x.size(1), x.size(2)};
  const Rows xr = rows(a[3], type, dev, "x", shape);
  const int32_t* positions = ints(a[2], dev, "positions", {tokens});
  const int inverse = PyObject_IsTrue(a[5]);
  if (inverse < 0) raise_set();
  Out out = a[6] == Py_None ? Out(make(shape, type, dev)) : Out(a[6]);
  const Rows yr = rows(out.o, type, dev, "out", shape);
  check(lla_rope_apply(&cfg, table.p, table.positions, layout_of(a[4]), inverse, kind, tokens,
                       small(shape[1], "x"), positions, xr.p, xr.stride, yr.p, yr.stride,
                       status_of(a[7], dev), stream_of(dev)));
  return out.release();
  END_HANDLE_TH_ERRORS
}

// (page, ctx_len, n_new, block_table, free_list, n_free, tok_cap, tok_start, slot, positions,
//  status) -> (tok_start, slot, positions)
PyObject* page_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 11);
  const c10::Device dev = leading(a[1], "ctx_len").device();
  const c10::cuda::CUDAGuard guard(dev);
  const Pages bt = pages_of(a[3], dev);
  const at::Tensor& fl = tensor(a[4], "free_list");
  if (fl.dim() != 1) fail(PyExc_ValueError, "free_list must be [n_pages]");
  const int64_t cap = integer(a[6]), B = bt.B;
  if (cap < 0) fail(PyExc_ValueError, "tok_cap must be >= 0");
  Out start = a[7] == Py_None ? Out(make({B + 1}, at::kInt, dev)) : Out(a[7]);
  Out slot = a[8] == Py_None ? Out(make({cap}, at::kLong, dev)) : Out(a[8]);
  Out positions = a[9] == Py_None ? Out(make({cap}, at::kInt, dev)) : Out(a[9]);
  int32_t* ctx = ints(a[1], dev, "ctx_len", {B});
  const int32_t* fresh = ints(a[2], dev, "n_new", {B});
  int32_t* list = dense<int32_t>(a[4], at::kInt, dev, "free_list");
  int32_t* n_free = ints(a[5], dev, "n_free", {1});
  check(lla_page_map((int32_t)B, integer32(a[0], "page"), bt.max_pages,
                     small(fl.size(0), "free_list"), ctx, fresh, bt.p, list, n_free, cap,
                     ints(start.o, dev, "tok_start", {B + 1}),
                     dense<int64_t>(slot.o, at::kLong, dev, "slot", {cap}),
                     ints(positions.o, dev, "positions", {cap}), status_of(a[10], dev),
                     stream_of(dev)));
  PyObject* r = PyTuple_New(3);
  if (!r) raise_set();
  PyTuple_SET_ITEM(r, 0, start.release());
  PyTuple_SET_ITEM(r, 1, slot.release());
  PyTuple_SET_ITEM(r, 2, positions.release());
  return r;
  END_HANDLE_TH_ERRORS
}

// (cfg, rope, cache, ctx_len, block_table, tok_start, positions, k, v, layout, status, row_start)
PyObject* q8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 12);
  const lla_cfg cfg = config(a[0]);
  const at::Tensor& k = leading(a[7], "k");
  const int kind = row_type(k, "k");
  const ScalarType type = k.scalar_type();
  const c10::Device dev = k.device();
  const c10::cuda::CUDAGuard guard(dev);
  const Pages bt = pages_of(a[4], dev);
  const Table table = table_of(a[1], cfg, dev);
  const lla_q8_cache cache = cache_of(a[2], cfg, dev);
  if (k.dim() != 3) fail(PyExc_ValueError, "k must be [tokens, heads, d]");
  const int64_t tokens = k.size(0), shape[] = {tokens, cfg.H, cfg.d_head};
  const Rows kr = rows(a[7], type, dev, "k", shape), vr = rows(a[8], type, dev, "v", shape);
  const int32_t* positions =
      a[6] == Py_None ? nullptr : ints(a[6], dev, "positions", {tokens});
  const int32_t* row_start =
      a[11] == Py_None ? nullptr : ints(a[11], dev, "row_start", {bt.B});
  check(lla_q8_append_rows(&cfg, &cache, table.p, table.positions, layout_of(a[9]), kind, bt.B,
                           bt.max_pages, ints(a[3], dev, "ctx_len", {bt.B}), bt.p,
                           small(tokens, "k"), ints(a[5], dev, "tok_start", {bt.B + 1}), positions,
                           row_start, kr.p, kr.stride, vr.p, vr.stride, status_of(a[10], dev),
                           stream_of(dev)));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (cfg, cache, slot, k_out, v_out, status) -> (k_out, v_out)
PyObject* q8_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 6);
  const lla_cfg cfg = config(a[0]);
  const at::Tensor& slot = leading(a[2], "slot");
  const c10::Device dev = slot.device();
  const c10::cuda::CUDAGuard guard(dev);
  const lla_q8_cache cache = cache_of(a[1], cfg, dev);
  if (slot.dim() != 1) fail(PyExc_ValueError, "slot must be [rows]");
  const int64_t shape[] = {slot.size(0), cfg.H, cfg.d_head};
  const at::TensorOptions opt = at::TensorOptions().dtype(at::kBFloat16).device(dev);
  const int64_t* slots = dense<int64_t>(a[2], at::kLong, dev, "slot");
  Out k = a[3] == Py_None ? Out(at::zeros(shape, opt)) : Out(a[3]);
  Out v = a[4] == Py_None ? Out(at::zeros(shape, opt)) : Out(a[4]);
  check(lla_q8_read(&cfg, &cache, shape[0], slots,
                    dense<uint16_t>(k.o, at::kBFloat16, dev, "k_out", shape),
                    dense<uint16_t>(v.o, at::kBFloat16, dev, "v_out", shape),
                    status_of(a[5], dev), stream_of(dev)));
  return PyTuple_Pack(2, k.o, v.o);
  END_HANDLE_TH_ERRORS
}

// (cfg, rope, cache, ctx_len, block_table, q, k_self, v_self, q_pos, layout, out, ws) -> out
PyObject* q8_decode_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 12);
  const lla_cfg cfg = config(a[0]);
  const at::Tensor& q = leading(a[5], "q");
  const int kind = row_type(q, "q");
  const ScalarType type = q.scalar_type();
  const c10::Device dev = q.device();
  const c10::cuda::CUDAGuard guard(dev);
  const Pages bt = pages_of(a[4], dev);
  const Table table = table_of(a[1], cfg, dev);
  const lla_q8_cache cache = cache_of(a[2], cfg, dev);
  const int64_t shape[] = {bt.B, cfg.H, cfg.d_head};
  const void* qp = dense<void>(a[5], type, dev, "q", shape);
  const void* kp = a[6] == Py_None ? nullptr : dense<void>(a[6], type, dev, "k_self", shape);
  const void* vp = a[7] == Py_None ? nullptr : dense<void>(a[7], type, dev, "v_self", shape);
  const int32_t* q_pos = a[8] == Py_None ? nullptr : ints(a[8], dev, "q_pos", {bt.B});
  const int32_t* ctx = ints(a[3], dev, "ctx_len", {bt.B});
  const int layout = layout_of(a[9]);
  Out out = a[10] == Py_None ? Out(make(shape, type, dev)) : Out(a[10]);
  void* op = dense<void>(out.o, type, dev, "out", shape);
  at::Tensor own;                 // without ws: zeros for this call
  void* ws;
  size_t bytes;
  if (a[11] == Py_None) {
    const int64_t cap = (int64_t)bt.max_pages * cache.page;
    bytes = lla_q8_decode_workspace_bytes(&cfg, bt.B, small(cap, "block_table"));
    if (!bytes) check(LLA_ERR_UNSUPPORTED);
    own = at::zeros({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
    ws = own.data_ptr();
  } else {
    ws = dense<void>(a[11], at::kByte, dev, "ws");
    bytes = THPVariable_Unpack(a[11]).numel();
  }
  check(lla_q8_decode_attn(&cfg, &cache, table.p, table.positions, layout, kind, bt.B,
                           bt.max_pages, ctx, bt.p, qp, kp, vp, q_pos, op, ws, bytes,
                           stream_of(dev)));
  return out.release();
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"rope_apply", method(rope_apply), METH_FASTCALL, nullptr},
    {"page_map", method(page_map), METH_FASTCALL, nullptr},
    {"q8_append", method(q8_append), METH_FASTCALL, nullptr},
    {"q8_read", method(q8_read), METH_FASTCALL, nullptr},
    {"q8_decode_attn", method(q8_decode_attn), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  static const char* names[] = {"T", "H", "d_head", "r_k", "r_v", "mode", "d_rope", "rope_base",
                                "sm_scale", "k", "v", "k_scale", "v_scale"};
  for (int i = 0; i < 13; ++i)
    if (!(g_names[i] = PyUnicode_InternFromString(names[i]))) return nullptr;
  return PyModule_Create(&g_module);
}
