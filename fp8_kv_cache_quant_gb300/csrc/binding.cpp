// The compiled part of the Python binding: argument checks and the calls of the entry points whose
// small calls are bound by the host (the rotary cache writes and the attention over block-scaled
// caches).  A decode step makes these calls once per layer, and their kernels run for a few
// microseconds; checking a dozen tensors' types, shapes and devices takes Python ten.
//
// Every function takes the raw stream, then its arguments in order (None for an absent tensor),
// raises ValueError for a tensor that does not fit and returns (status, result tensor or None).
// The tensors' device must be current.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "../../include/fp8kv.h"

namespace {

using at::Tensor;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* fn, const std::string& what) {
  PyErr_SetString(PyExc_ValueError, (std::string(fn) + ": " + what).c_str());
  throw Refused();
}

// The arguments of one call, taken in order.
struct Args {
  const char* fn;
  PyObject* const* a;
  Py_ssize_t n, i = 0;

  PyObject* next() {
    if (i >= n) refuse(fn, "too few arguments");
    return a[i++];
  }
  long long integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
  }
  int32_t i32() {
    const long long v = integer();
    if (v < INT32_MIN || v > INT32_MAX) refuse(fn, "an integer beyond 32 bits");
    return static_cast<int32_t>(v);
  }
  float real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return static_cast<float>(v);
  }
  void* pointer() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    void* v = PyLong_AsVoidPtr(o);
    if (v == nullptr && PyErr_Occurred()) throw Refused();
    return v;
  }
  // an absent tensor (None) is undefined
  Tensor tensor(const char* name, bool may_be_none = false) {
    PyObject* o = next();
    if (o == Py_None && may_be_none) return Tensor();
    if (!THPVariable_Check(o)) refuse(fn, std::string(name) + " is not a tensor");
    return THPVariable_Unpack(o);
  }
  void done() {
    if (i != n) refuse(fn, "too many arguments");
  }
};

std::string text(at::IntArrayRef shape) {
  std::string s = "[";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "]";
}

std::string text(const Tensor& t) {
  return std::string(c10::toString(t.scalar_type())) + " " + text(t.sizes()) + " on " + t.device().str();
}

// A contiguous tensor of that type and shape on the device; its address (null when undefined).
template <typename T = void>
T* fits(const char* fn, const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  if (!t.defined()) return nullptr;
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != device || !t.is_contiguous())
    refuse(fn, std::string(name) + " is " + text(t) + (t.is_contiguous() ? "" : ", not contiguous") + "; wanted " +
                   c10::toString(type) + " " + text(shape) + " on " + device.str() + ", contiguous");
  return static_cast<T*>(t.data_ptr());
}

// The token stride of a bf16 tensor [n][heads][d] whose rows are consecutive (a slice of a wider
// projection's output serves).
int64_t row_stride(const char* fn, const char* name, const Tensor& t, int64_t n, int64_t heads, int64_t d, at::Device device) {
  const int64_t shape[3] = {n, heads, d};
  if (t.scalar_type() != at::kBFloat16 || t.sizes() != at::IntArrayRef(shape, 3) || t.device() != device)
    refuse(fn, std::string(name) + " is " + text(t) + "; wanted BFloat16 " + text(at::IntArrayRef(shape, 3)) + " on " + device.str());
  if (n == 0) return heads * d;
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
    refuse(fn, std::string(name) + "'s rows are not consecutive (strides " + text(t.strides()) + ")");
  return n > 1 ? t.stride(0) : heads * d;
}

int32_t small(const char* fn, int64_t v) {
  if (v < 0 || v > INT32_MAX) refuse(fn, "a size beyond 32 bits");
  return static_cast<int32_t>(v);
}

Tensor three_dims(Args& a, const char* name) {
  Tensor t = a.tensor(name);
  if (t.dim() != 3) refuse(a.fn, std::string(name) + " is " + text(t) + "; wanted [n][heads][head_dim]");
  return t;
}

// Optional queries [n][Hq][d] and where they go.
struct Queries {
  Tensor q, out;
  const void* src = nullptr;
  void* dst = nullptr;
  int64_t stride = 0, out_stride = 0;
  int32_t heads = 0;

  void check(const char* fn, int64_t n, int64_t d, at::Device device) {
    if (!q.defined()) {
      if (out.defined()) refuse(fn, "q_out without q");
      return;
    }
    if (q.dim() != 3) refuse(fn, "q is " + text(q) + "; wanted [n][heads][head_dim]");
    heads = small(fn, q.size(1));
    stride = row_stride(fn, "q", q, n, heads, d, device);
    if (!out.defined()) out = at::empty({n, heads, d}, q.options());
    out_stride = row_stride(fn, "q_out", out, n, heads, d, device);
    src = q.data_ptr();
    dst = out.data_ptr();
  }
};

fkv_rope rope_of(const char* fn, const Tensor& cos_sin, bool interleaved, at::Device device) {
  fkv_rope r = {nullptr, 0, 0, 0};
  if (!cos_sin.defined()) return r;
  if (cos_sin.dim() != 2) refuse(fn, "cos_sin is " + text(cos_sin) + "; wanted [positions][rot_dim]");
  r.cos_sin = fits<float>(fn, "cos_sin", cos_sin, at::kFloat, cos_sin.sizes(), device);
  r.max_positions = small(fn, cos_sin.size(0));
  r.rot_dim = small(fn, cos_sin.size(1));
  r.interleaved = interleaved;
  return r;
}

// The next four arguments, a block-scaled cache whose heads are `heads` (-1: any) by d.
fkv_block_cache block_cache(Args& a, int64_t heads, int64_t d, at::Device device) {
  const Tensor k = a.tensor("k_cache"), v = a.tensor("v_cache"), ks = a.tensor("k_scale"), vs = a.tensor("v_scale");
  if (k.dim() != 4) refuse(a.fn, "k_cache is " + text(k) + "; wanted [blocks][heads][16][head_dim]");
  const int64_t nb = k.size(0), h = heads < 0 ? k.size(1) : heads, bs = k.size(2);
  fkv_block_cache c;
  c.k_cache = fits(a.fn, "k_cache", k, at::kByte, {nb, h, bs, d}, device);
  c.v_cache = fits(a.fn, "v_cache", v, at::kByte, {nb, h, bs, d}, device);
  c.k_scale = fits<float>(a.fn, "k_scale", ks, at::kFloat, {nb, h}, device);
  c.v_scale = fits<float>(a.fn, "v_scale", vs, at::kFloat, {nb, h}, device);
  c.num_blocks = small(a.fn, nb);
  c.block_size = small(a.fn, bs);
  c.num_kv_heads = small(a.fn, h);
  c.head_dim = small(a.fn, d);
  return c;
}

PyObject* result(fkv_status st, const Tensor& t) {
  PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
  return Py_BuildValue("iN", static_cast<int>(st), o);
}

// stream, q, k, v, positions, slot_mapping, cos_sin, interleaved, k_cache, v_cache, kv_format,
// k_scale, v_scale, gran, layer, mask address, its length, whether the layer is skipped, q_out, fault
PyObject* kv_rope_cache_(Args a) {
  void* stream = a.pointer();
  Queries q;
  q.q = a.tensor("q", true);
  const Tensor k = three_dims(a, "k"), v = a.tensor("v"), pos = a.tensor("positions"), slots = a.tensor("slot_mapping"),
               cs = a.tensor("cos_sin");
  const bool interleaved = a.integer() != 0;
  const Tensor kc = a.tensor("k_cache"), vc = a.tensor("v_cache");
  fkv_layer_cache c;
  c.kv_format = a.i32();
  const Tensor ks = a.tensor("k_scale", true), vs = a.tensor("v_scale", true);
  const int32_t gran = a.i32(), layer = a.i32();
  const void* mask = a.pointer();
  const int32_t layers = a.i32();
  const at::ScalarType type = a.integer() ? at::kBFloat16 : at::kByte;
  q.out = a.tensor("q_out", true);
  const Tensor fault = a.tensor("fault", true);
  a.done();
  const at::Device dev = k.device();
  const int64_t n = k.size(0), h = k.size(1), d = k.size(2);
  const int64_t k_stride = row_stride(a.fn, "k", k, n, h, d, dev), v_stride = row_stride(a.fn, "v", v, n, h, d, dev);
  q.check(a.fn, n, d, dev);
  if (kc.dim() != 4) refuse(a.fn, "k_cache is " + text(kc) + "; wanted [blocks][heads][16][head_dim]");
  const int64_t nb = kc.size(0), bs = kc.size(2), scales = gran == FKV_SCALE_PER_HEAD ? h : 1;
  c.k_cache = fits(a.fn, "k_cache", kc, type, {nb, h, bs, d}, dev);
  c.v_cache = fits(a.fn, "v_cache", vc, type, {nb, h, bs, d}, dev);
  c.num_blocks = small(a.fn, nb);
  c.block_size = small(a.fn, bs);
  c.num_kv_heads = small(a.fn, h);
  c.head_dim = small(a.fn, d);
  const fkv_status st = kv_rope_cache(
      q.src, q.stride, q.dst, q.out_stride, q.heads, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
      fits<int64_t>(a.fn, "positions", pos, at::kLong, {n}, dev), fits<int64_t>(a.fn, "slot_mapping", slots, at::kLong, {n}, dev),
      small(a.fn, n), rope_of(a.fn, cs, interleaved, dev), c, fits<float>(a.fn, "k_scale", ks, at::kFloat, {scales}, dev),
      fits<float>(a.fn, "v_scale", vs, at::kFloat, {scales}, dev), static_cast<fkv_scale_gran>(gran), layer,
      static_cast<const uint8_t*>(mask), layers, fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev),
      static_cast<fkv_stream_t>(stream));
  return result(st, q.out);
}

// stream, k, v, cu_seqlens, max_q_len, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, cos_sin,
// interleaved, q, q_out, fault
PyObject* kv_block_cache_(Args a) {
  void* stream = a.pointer();
  const Tensor k = three_dims(a, "k"), v = a.tensor("v"), cu = a.tensor("cu_seqlens");
  const int32_t max_q_len = a.i32();
  const at::Device dev = k.device();
  const int64_t n = k.size(0), h = k.size(1), d = k.size(2);
  const fkv_block_cache c = block_cache(a, h, d, dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens"), cs = a.tensor("cos_sin", true);
  const bool interleaved = a.integer() != 0;
  Queries q;
  q.q = a.tensor("q", true);
  q.out = a.tensor("q_out", true);
  const Tensor fault = a.tensor("fault", true);
  a.done();
  const int64_t k_stride = row_stride(a.fn, "k", k, n, h, d, dev), v_stride = row_stride(a.fn, "v", v, n, h, d, dev);
  q.check(a.fn, n, d, dev);
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  const int64_t b = table.size(0);
  const fkv_status st = kv_block_cache(
      q.src, q.stride, q.dst, q.out_stride, q.heads, k.data_ptr(), k_stride, v.data_ptr(), v_stride, small(a.fn, n),
      fits<int32_t>(a.fn, "cu_seqlens", cu, at::kInt, {b + 1}, dev), small(a.fn, b), max_q_len,
      rope_of(a.fn, cs, interleaved, dev), c, fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev),
      small(a.fn, table.size(1)), fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev),
      fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev), static_cast<fkv_stream_t>(stream));
  return result(st, q.out);
}

// stream, q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, softmax_scale, window, out, workspace, fault
PyObject* fp8_block_decode_attn_(Args a) {
  void* stream = a.pointer();
  const Tensor q = three_dims(a, "q");
  const at::Device dev = q.device();
  const fkv_block_cache c = block_cache(a, -1, q.size(2), dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens");
  const float softmax_scale = a.real();
  const int32_t window = a.i32();
  Tensor out = a.tensor("out", true);
  const Tensor workspace = a.tensor("workspace");
  const Tensor fault = a.tensor("fault", true);
  a.done();
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  const int64_t b = table.size(0), hq = q.size(1), d = q.size(2);
  const void* src = fits(a.fn, "q", q, at::kBFloat16, {b, hq, d}, dev);
  if (!out.defined()) out = at::empty({b, hq, d}, q.options());
  if (workspace.device() != dev || !workspace.is_contiguous()) refuse(a.fn, "workspace is " + text(workspace) + "; wanted contiguous on " + dev.str());
  const fkv_status st = fp8_block_decode_attn(
      src, small(a.fn, b), small(a.fn, hq), c,
      fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev), small(a.fn, table.size(1)),
      fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev), softmax_scale, window,
      fits(a.fn, "out", out, at::kBFloat16, {b, hq, d}, dev), workspace.data_ptr(), workspace.nbytes(),
      fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev), static_cast<fkv_stream_t>(stream));
  return result(st, out);
}

// stream, q, cu_seqlens_q, max_q_len, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, softmax_scale,
// causal, window, out, fault
PyObject* fp8_block_prefill_attn_(Args a) {
  void* stream = a.pointer();
  const Tensor q = three_dims(a, "q"), cu = a.tensor("cu_seqlens_q");
  const int32_t max_q_len = a.i32();
  const at::Device dev = q.device();
  const fkv_block_cache c = block_cache(a, -1, q.size(2), dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens");
  const float softmax_scale = a.real();
  const int32_t causal = a.integer() != 0, window = a.i32();
  Tensor out = a.tensor("out", true);
  const Tensor fault = a.tensor("fault", true);
  a.done();
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  const int64_t b = table.size(0);
  const void* src = fits(a.fn, "q", q, at::kBFloat16, q.sizes(), dev);
  if (!out.defined()) out = at::empty(q.sizes(), q.options());
  const fkv_status st = fp8_block_prefill_attn(
      src, fits<int32_t>(a.fn, "cu_seqlens_q", cu, at::kInt, {b + 1}, dev),
      small(a.fn, q.size(0)), small(a.fn, b), small(a.fn, q.size(1)), max_q_len, c,
      fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev), small(a.fn, table.size(1)),
      fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev), softmax_scale, causal, window,
      fits(a.fn, "out", out, at::kBFloat16, q.sizes(), dev), fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev),
      static_cast<fkv_stream_t>(stream));
  return result(st, out);
}

// No C++ exception leaves a call: what torch throws becomes a RuntimeError.
template <PyObject* (*kBody)(Args)>
PyObject* entry(const char* fn, PyObject* const* args, Py_ssize_t n) {
  try {
    return kBody(Args{fn, args, n});
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

#define FKV_ENTRY(name)                                                                                           \
  PyObject* name##_py(PyObject*, PyObject* const* args, Py_ssize_t n) { return entry<name##_>(#name, args, n); }
FKV_ENTRY(kv_rope_cache)
FKV_ENTRY(kv_block_cache)
FKV_ENTRY(fp8_block_decode_attn)
FKV_ENTRY(fp8_block_prefill_attn)
#undef FKV_ENTRY

#define FKV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name##_py)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FKV_METHOD(kv_rope_cache), FKV_METHOD(kv_block_cache), FKV_METHOD(fp8_block_decode_attn),
                         FKV_METHOD(fp8_block_prefill_attn), {nullptr, nullptr, 0, nullptr}};
#undef FKV_METHOD

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Checked calls of libfp8kv.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
