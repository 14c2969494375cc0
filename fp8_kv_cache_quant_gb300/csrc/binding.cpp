// The compiled part of the Python binding: argument checks and the calls of the entry points whose
// small calls are bound by the host (the rotary cache writes, and the attention over block-scaled
// caches with its weights and the eviction).  A decode step makes these calls once per layer, and their kernels run for a few
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

// The axes of a rope's pairs, two arguments (the address of their bytes, null for none, and their number), and the
// positions of n tokens that go with them: int64 [n], or [axes][n] whose rows may be slices.
struct Axes {
  const uint8_t* pair;
  int64_t pairs;

  Axes(Args& a, bool given) : pair(given ? static_cast<const uint8_t*>(a.pointer()) : nullptr), pairs(given ? a.integer() : 0) {}
  fkv_axes of(const char* fn, const Tensor& pos, int64_t n, const fkv_rope& rope, at::Device device) const {
    fkv_axes x = {nullptr, 0, 1, pair};
    if (pair && pairs != rope.rot_dim / 2) refuse(fn, "the rope names the axes of " + std::to_string(pairs) + " pairs; its table has " + std::to_string(rope.rot_dim / 2));
    if (!pair) {
      x.positions = fits<int64_t>(fn, "positions", pos, at::kLong, {n}, device);
      return x;
    }
    if (pos.scalar_type() != at::kLong || pos.dim() != 2 || pos.size(1) != n || pos.device() != device || (n > 1 && pos.stride(1) != 1))
      refuse(fn, "positions is " + text(pos) + "; wanted Long [axes, " + std::to_string(n) + "] on " + device.str() + " with consecutive rows");
    x.positions = static_cast<const int64_t*>(pos.data_ptr());
    x.num_axes = small(fn, pos.size(0));
    x.axis_stride = pos.stride(0);
    return x;
  }
};

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

// stream, q, k, v, positions, slot_mapping, cos_sin, interleaved, kAxes: the pairs' axes (see Axes), k_cache, v_cache, kv_format,
// k_scale, v_scale, gran, layer, mask address, its length, whether the layer is skipped, q_out, fault
template <bool kAxes>
PyObject* rope_cache(Args a) {
  void* stream = a.pointer();
  Queries q;
  q.q = a.tensor("q", true);
  const Tensor k = three_dims(a, "k"), v = a.tensor("v"), pos = a.tensor("positions"), slots = a.tensor("slot_mapping"),
               cs = a.tensor("cos_sin");
  const bool interleaved = a.integer() != 0;
  const Axes axes(a, kAxes);
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
  const fkv_rope rope = rope_of(a.fn, cs, interleaved, dev);
  const fkv_status st = kv_rope_cache_axes(
      q.src, q.stride, q.dst, q.out_stride, q.heads, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
      axes.of(a.fn, pos, n, rope, dev), fits<int64_t>(a.fn, "slot_mapping", slots, at::kLong, {n}, dev),
      small(a.fn, n), rope, c, fits<float>(a.fn, "k_scale", ks, at::kFloat, {scales}, dev),
      fits<float>(a.fn, "v_scale", vs, at::kFloat, {scales}, dev), static_cast<fkv_scale_gran>(gran), layer,
      static_cast<const uint8_t*>(mask), layers, fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev),
      static_cast<fkv_stream_t>(stream));
  return result(st, q.out);
}

// stream, k, v, cu_seqlens, max_q_len, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, cos_sin,
// interleaved, kAxes: the pairs' axes (see Axes) and positions, q, q_out, fault
template <bool kAxes>
PyObject* block_cache_append(Args a) {
  void* stream = a.pointer();
  const Tensor k = three_dims(a, "k"), v = a.tensor("v"), cu = a.tensor("cu_seqlens");
  const int32_t max_q_len = a.i32();
  const at::Device dev = k.device();
  const int64_t n = k.size(0), h = k.size(1), d = k.size(2);
  const fkv_block_cache c = block_cache(a, h, d, dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens"), cs = a.tensor("cos_sin", true);
  const bool interleaved = a.integer() != 0;
  const Axes axes(a, kAxes);
  const Tensor pos = kAxes ? a.tensor("positions") : Tensor();
  Queries q;
  q.q = a.tensor("q", true);
  q.out = a.tensor("q_out", true);
  const Tensor fault = a.tensor("fault", true);
  a.done();
  const int64_t k_stride = row_stride(a.fn, "k", k, n, h, d, dev), v_stride = row_stride(a.fn, "v", v, n, h, d, dev);
  q.check(a.fn, n, d, dev);
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  const int64_t b = table.size(0);
  const fkv_rope rope = rope_of(a.fn, cs, interleaved, dev);
  const int32_t *starts = fits<int32_t>(a.fn, "cu_seqlens", cu, at::kInt, {b + 1}, dev),
                *blocks = fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev),
                *lens = fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev);
  int32_t* const flt = fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev);
  const auto call = [&](auto entry, auto... positions) {
    return entry(q.src, q.stride, q.dst, q.out_stride, q.heads, k.data_ptr(), k_stride, v.data_ptr(), v_stride, small(a.fn, n),
                 positions..., starts, small(a.fn, b), max_q_len, rope, c, blocks, small(a.fn, table.size(1)), lens, flt,
                 static_cast<fkv_stream_t>(stream));
  };
  if (!kAxes) return result(call(kv_block_cache), q.out);
  if (!cs.defined()) refuse(a.fn, "positions without a rope");
  return result(call(kv_block_cache_axes, axes.of(a.fn, pos, n, rope, dev)), q.out);
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

// stream, q, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, group_starts, shared_lens, softmax_scale, window, out,
// workspace, fault
PyObject* fp8_block_shared_decode_attn_(Args a) {
  void* stream = a.pointer();
  const Tensor q = three_dims(a, "q");
  const at::Device dev = q.device();
  const fkv_block_cache c = block_cache(a, -1, q.size(2), dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens"), starts = a.tensor("group_starts"), shared = a.tensor("shared_lens");
  const float softmax_scale = a.real();
  const int32_t window = a.i32();
  Tensor out = a.tensor("out", true);
  const Tensor workspace = a.tensor("workspace"), fault = a.tensor("fault", true);
  a.done();
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  if (shared.dim() != 1) refuse(a.fn, "shared_lens is " + text(shared) + "; wanted [groups]");
  const int64_t b = table.size(0), hq = q.size(1), d = q.size(2), n = shared.size(0);
  const void* src = fits(a.fn, "q", q, at::kBFloat16, {b, hq, d}, dev);
  if (!out.defined()) out = at::empty({b, hq, d}, q.options());
  if (workspace.device() != dev || !workspace.is_contiguous()) refuse(a.fn, "workspace is " + text(workspace) + "; wanted contiguous on " + dev.str());
  const fkv_status st = fp8_block_shared_decode_attn(
      src, small(a.fn, b), small(a.fn, hq), c, fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev),
      small(a.fn, table.size(1)), fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev),
      fits<int32_t>(a.fn, "group_starts", starts, at::kInt, {n + 1}, dev), fits<int32_t>(a.fn, "shared_lens", shared, at::kInt, {n}, dev),
      small(a.fn, n), softmax_scale, window, fits(a.fn, "out", out, at::kBFloat16, {b, hq, d}, dev), workspace.data_ptr(),
      workspace.nbytes(), fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev), static_cast<fkv_stream_t>(stream));
  return result(st, out);
}

// stream, q, cu_seqlens_q, max_q_len, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, weights, softmax_scale,
// decay, workspace, fault
PyObject* fp8_block_attn_weights_(Args a) {
  void* stream = a.pointer();
  const Tensor q = three_dims(a, "q"), cu = a.tensor("cu_seqlens_q");
  const int32_t max_q_len = a.i32();
  const at::Device dev = q.device();
  const fkv_block_cache c = block_cache(a, -1, q.size(2), dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens"), weights = a.tensor("weights");
  const float softmax_scale = a.real(), decay = a.real();
  const Tensor workspace = a.tensor("workspace"), fault = a.tensor("fault", true);
  a.done();
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  if (weights.dim() != 3) refuse(a.fn, "weights is " + text(weights) + "; wanted [batch][heads][tokens]");
  const int64_t b = table.size(0), len = weights.size(2);
  if (workspace.device() != dev || !workspace.is_contiguous()) refuse(a.fn, "workspace is " + text(workspace) + "; wanted contiguous on " + dev.str());
  const void* src = fits(a.fn, "q", q, at::kBFloat16, q.sizes(), dev);
  const fkv_status st = fp8_block_attn_weights(
      src, fits<int32_t>(a.fn, "cu_seqlens_q", cu, at::kInt, {b + 1}, dev), small(a.fn, q.size(0)), small(a.fn, b),
      small(a.fn, q.size(1)), max_q_len, c, fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev),
      small(a.fn, table.size(1)), fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev), softmax_scale, decay,
      fits<float>(a.fn, "weights", weights, at::kFloat, {b, c.num_kv_heads, len}, dev), small(a.fn, len), workspace.data_ptr(),
      workspace.nbytes(), fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev), static_cast<fkv_stream_t>(stream));
  return result(st, weights);
}

// stream, k_cache, v_cache, k_scale, v_scale, block_table, context_lens, weights, budget, sink, recent, new_table, new_weights,
// new_lens, kept, fault
PyObject* kv_block_evict_(Args a) {
  void* stream = a.pointer();
  const Tensor kc = a.tensor("k_cache");
  --a.i;
  if (kc.dim() != 4) refuse(a.fn, "k_cache is " + text(kc) + "; wanted [blocks][heads][16][head_dim]");
  const at::Device dev = kc.device();
  const fkv_block_cache c = block_cache(a, -1, kc.size(3), dev);
  const Tensor table = a.tensor("block_table"), ctx = a.tensor("context_lens"), weights = a.tensor("weights");
  const int32_t budget = a.i32(), sink = a.i32(), recent = a.i32();
  const Tensor new_table = a.tensor("new_table"), new_weights = a.tensor("new_weights", true), new_lens = a.tensor("new_lens"),
               kept = a.tensor("kept"), fault = a.tensor("fault", true);
  a.done();
  if (table.dim() != 2) refuse(a.fn, "block_table is " + text(table) + "; wanted [batch][blocks]");
  if (new_table.dim() != 2) refuse(a.fn, "new_table is " + text(new_table) + "; wanted [batch][blocks]");
  if (weights.dim() != 3) refuse(a.fn, "weights is " + text(weights) + "; wanted [batch][heads][tokens]");
  if (new_weights.defined() && new_weights.dim() != 3) refuse(a.fn, "new_weights is " + text(new_weights) + "; wanted [batch][heads][tokens]");
  const int64_t b = table.size(0), h = c.num_kv_heads, len = weights.size(2), new_len = new_weights.defined() ? new_weights.size(2) : 0;
  const fkv_status st = kv_block_evict(
      c, fits<int32_t>(a.fn, "block_table", table, at::kInt, table.sizes(), dev), small(a.fn, b), small(a.fn, table.size(1)),
      fits<int32_t>(a.fn, "context_lens", ctx, at::kInt, {b}, dev), fits<float>(a.fn, "weights", weights, at::kFloat, {b, h, len}, dev),
      small(a.fn, len), budget, sink, recent, fits<int32_t>(a.fn, "new_table", new_table, at::kInt, {b, new_table.size(1)}, dev),
      small(a.fn, new_table.size(1)), fits<int32_t>(a.fn, "new_lens", new_lens, at::kInt, {b}, dev),
      fits<int32_t>(a.fn, "kept", kept, at::kInt, {b, h, budget}, dev),
      fits<float>(a.fn, "new_weights", new_weights, at::kFloat, {b, h, new_len}, dev), small(a.fn, new_len),
      fits<int32_t>(a.fn, "fault", fault, at::kInt, {1}, dev), static_cast<fkv_stream_t>(stream));
  return result(st, Tensor());
}

PyObject* kv_rope_cache_(Args a) { return rope_cache<false>(a); }
PyObject* kv_rope_cache_axes_(Args a) { return rope_cache<true>(a); }
PyObject* kv_block_cache_(Args a) { return block_cache_append<false>(a); }
PyObject* kv_block_cache_axes_(Args a) { return block_cache_append<true>(a); }

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
FKV_ENTRY(kv_rope_cache_axes)
FKV_ENTRY(kv_block_cache_axes)
FKV_ENTRY(kv_block_evict)
FKV_ENTRY(fp8_block_shared_decode_attn)
FKV_ENTRY(fp8_block_attn_weights)
FKV_ENTRY(fp8_block_decode_attn)
FKV_ENTRY(fp8_block_prefill_attn)
#undef FKV_ENTRY

#define FKV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name##_py)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FKV_METHOD(kv_rope_cache), FKV_METHOD(kv_block_cache), FKV_METHOD(kv_rope_cache_axes),
                         FKV_METHOD(kv_block_cache_axes), FKV_METHOD(kv_block_evict), FKV_METHOD(fp8_block_shared_decode_attn),
                         FKV_METHOD(fp8_block_attn_weights), FKV_METHOD(fp8_block_decode_attn),
                         FKV_METHOD(fp8_block_prefill_attn), {nullptr, nullptr, 0, nullptr}};
#undef FKV_METHOD

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Checked calls of libfp8kv.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
