// gdn_torch.cpp -- the Python binding of the operators around the recurrence
// (norms, rotary positions, the paged 8-bit cache, attention of packed sequences,
// activations in 8 bits): argument checks, output allocation and the call of the C ABI, for PyTorch tensors.
//
// These operators take 1 to 4 us on the GPU for a decode step, and a binding in
// Python took 9 to 23 us of the host a call (checks of up to nine tensors, the
// outputs' allocation, the marshalling of up to 27 arguments).  This module does
// the same in a few microseconds.  It computes nothing: every step runs in
// libgdn's kernels.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <string>
#include <vector>

#include "../../include/gdn.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;  // GDNError(function, status)
PyObject *g_memory_error = nullptr;  // torch.OutOfMemoryError

struct Refused {  // a Python exception to raise
  PyObject *type;
  std::string text;
};
[[noreturn]] void type_error(const std::string &s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Refused{PyExc_ValueError, s}; }

std::string shape_text(const Tensor &t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}
const char *dtype_text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

// One call's arguments, taken in order.
struct Args {
  PyObject *const *v;
  Py_ssize_t n, i = 0;
  PyObject *next() {
    if (i >= n) type_error("too few arguments");
    return v[i++];
  }
  const Tensor &tensor(const char *name) {
    PyObject *o = next();
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
  }
  // An undefined tensor for None.
  const Tensor &maybe(const char *name) {
    static const Tensor none;
    if (i < n && v[i] == Py_None) {
      ++i;
      return none;
    }
    return tensor(name);
  }
  long long integer(const char *name) {
    const long long x = PyLong_AsLongLong(next());
    if (x == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      type_error(std::string(name) + " must be an integer");
    }
    return x;
  }
  int int32(const char *name) {
    const long long x = integer(name);
    if (x < -2147483648LL || x > 2147483647LL) value_error(std::string(name) + " does not fit 32 bits");
    return (int)x;
  }
  float real(const char *name) {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      type_error(std::string(name) + " must be a number");
    }
    return (float)x;
  }
};

// Makes the tensor's device the current one for the call: launches, and what the
// library asks of its device, go by that.
c10::cuda::CUDAGuard on_gpu(const Tensor &t, const char *name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be on a CUDA device, got " + t.device().str());
  return c10::cuda::CUDAGuard(t.device());
}
void kind(const Tensor &t, const char *name, at::ScalarType dtype, const at::Device &dev) {
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " must be " + dtype_text(dtype) + ", got " + dtype_text(t.scalar_type()));
  if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}
// A dense tensor of this type, device and number of dimensions (-1: any).
void need(const Tensor &t, const char *name, at::ScalarType dtype, const at::Device &dev, int64_t ndim) {
  kind(t, name, dtype, dev);
  if (ndim >= 0 && t.dim() != ndim)
    value_error(std::string(name) + " must have " + std::to_string(ndim) + " dims, got shape " + shape_text(t));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous (the library does not copy)");
}
// [T, heads, D] with dense heads and any token stride; returns that stride.
int64_t token_stride(const Tensor &t, const char *name, const at::Device &dev) {
  kind(t, name, at::kBFloat16, dev);
  if (t.dim() != 3) value_error(std::string(name) + " must have 3 dims, got shape " + shape_text(t));
  const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
  if ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1) || (T > 1 && t.stride(0) < H * D))
    value_error(std::string(name) + ": the heads of a token must be dense (the library does not copy)");
  return T > 1 ? t.stride(0) : H * D;
}
int fits32(int64_t x, const char *name) {
  if (x > 2147483647LL) value_error(std::string(name) + " does not fit 32 bits");
  return (int)x;
}
template <class T> T *ptr(const Tensor &t) { return t.defined() ? reinterpret_cast<T *>(t.data_ptr()) : nullptr; }
const uint16_t *bf(const Tensor &t) { return ptr<const uint16_t>(t); }
uint16_t *bf_out(const Tensor &t) { return ptr<uint16_t>(t); }
void *stream_of(const at::Device &d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }
Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) {
  return Tensor(at::detail::empty_cuda(shape, dtype, dev, std::nullopt));
}

struct Status {
  const char *fn;
  int code;
};
void done(const char *fn, int rc) {
  if (rc != GDN_OK) throw Status{fn, rc};
}
PyObject *wrap(const Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <int N> PyObject *tuple_of(const Tensor (&t)[N]) {
  PyObject *r = PyTuple_New(N);
  for (int i = 0; r && i < N; ++i) {
    PyObject *o = wrap(t[i]);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}
template <PyObject *(*F)(Args &)> PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n) {
  try {
    Args a{v, n};
    return F(a);
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Status &s) {
    PyObject *e = g_error ? PyObject_CallFunction(g_error, "si", s.fn, s.code) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s: status %d", s.fn, s.code);
    }
  } catch (const c10::OutOfMemoryError &e) {  // torch.OutOfMemoryError, as from torch's own calls
    PyErr_SetString(g_memory_error ? g_memory_error : PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ---------------------------------------------------------------- norms
struct Gate {
  int act;
  int64_t rows, stride;  // 0: dense
};
// Where the rows of a tensor lie: dense, or [.., heads, D] / [.., D] with one longer
// stride between its tokens.
Gate rows_of(const Tensor &z, const char *name, const char *fn) {
  if (z.is_contiguous()) return {0, 0, 0};
  // From the last dimension on: those that lie densely make a group (the heads of a
  // token), those before them one walk from group to group.
  int64_t i = z.dim() - 1, dense = 1, rows = 1;
  for (; i >= 0 && (z.size(i) == 1 || z.stride(i) == dense); --i) {
    if (i < z.dim() - 1) rows *= z.size(i);
    dense *= z.size(i);
  }
  const int64_t stride = i >= 0 ? z.stride(i) : dense;
  int64_t next = stride;
  bool even = i < z.dim() - 1;
  for (; i >= 0; --i) {
    even = even && (z.size(i) == 1 || z.stride(i) == next);
    next *= z.size(i);
  }
  if (!even) value_error(std::string(fn) + ": " + name + " must be dense, or [.., heads, D] / [.., D] with one longer stride between its tokens");
  return {0, rows, stride};
}
Gate gate_of(const Tensor &z, const Tensor &x, int act, const char *fn) {
  if (!z.defined()) return {0, 0, 0};
  if (act == 0) value_error(std::string(fn) + ": a gate z needs an activation");
  kind(z, "z", at::kBFloat16, x.device());
  if (z.sizes() != x.sizes()) value_error(std::string(fn) + ": z must have the shape of x, " + shape_text(x));
  const Gate g = rows_of(z, "z", fn);
  return {act, g.rows, g.stride};
}
void like(const Tensor &t, const char *name, const Tensor &x, const char *fn) {
  need(t, name, at::kBFloat16, x.device(), -1);
  if (t.sizes() != x.sizes()) value_error(std::string(fn) + ": " + name + " must have the shape " + shape_text(x));
}
int width_of(const Tensor &x, const Tensor &w, const char *fn) {
  need(w, "weight", at::kFloat, x.device(), 1);
  const int64_t D = x.dim() ? x.size(-1) : 0;
  if (D < 1 || w.size(0) != D)
    value_error(std::string(fn) + ": weight must be [D] for rows of D, got " + shape_text(w) + " and " + shape_text(x));
  return fits32(D, "D");
}

PyObject *norm_gate(Args &a) {
  const char *fn = "gdn_norm_gate";
  const Tensor &x = a.tensor("x"), &w = a.tensor("weight"), &res = a.maybe("residual"), &z = a.maybe("z");
  const int act = a.int32("activation");
  const float eps = a.real("eps"), rs = a.real("res_scale");
  Tensor y = a.maybe("y"), h = a.maybe("h");
  const auto device = on_gpu(x, "x");
  need(x, "x", at::kBFloat16, x.device(), -1);
  const int D = width_of(x, w, fn);
  const Gate g = gate_of(z, x, act, fn);
  if (y.defined()) like(y, "y", x, fn);
  else y = empty(x.sizes(), at::kBFloat16, x.device());
  if (res.defined()) {
    like(res, "residual", x, fn);
    if (h.defined()) like(h, "h", x, fn);
    else h = empty(x.sizes(), at::kBFloat16, x.device());
  } else if (h.defined()) {
    value_error("gdn_norm_gate: h is an output of the form with a residual");
  }
  done(fn, gdn_norm_gate(bf(x), bf(res), g.act ? bf(z) : nullptr, ptr<const float>(w), rs, eps, g.act, x.numel() / D, D, g.rows,
                         g.stride, bf_out(y), bf_out(h), stream_of(x.device())));
  const Tensor out[2] = {y, h};
  return tuple_of(out);
}

PyObject *norm_gate_bwd(Args &a) {
  const char *fn = "gdn_norm_gate_bwd";
  const Tensor &dy = a.tensor("dy"), &h = a.tensor("h"), &w = a.tensor("weight"), &z = a.maybe("z"), &dh = a.maybe("dh");
  const int act = a.int32("activation");
  const float eps = a.real("eps"), rs = a.real("res_scale");
  Tensor ws = a.maybe("workspace");
  const auto device = on_gpu(h, "h");
  need(h, "h", at::kBFloat16, h.device(), -1);
  like(dy, "dy", h, fn);
  const int D = width_of(h, w, fn);
  const Gate g = gate_of(z, h, act, fn);
  if (dh.defined()) like(dh, "dh", h, fn);
  const at::Device dev = h.device();
  const Tensor dx = empty(h.sizes(), at::kBFloat16, dev), dw = empty(w.sizes(), at::kFloat, dev);
  const Tensor dres = dh.defined() ? empty(h.sizes(), at::kBFloat16, dev) : Tensor();
  const Tensor dz = g.act ? empty(h.sizes(), at::kBFloat16, dev) : Tensor();
  const int64_t rows = h.numel() / D;
  if (ws.defined()) need(ws, "workspace", at::kByte, dev, 1);
  else ws = empty({(int64_t)gdn_norm_gate_bwd_workspace_size(rows, D)}, at::kByte, dev);
  done(fn, gdn_norm_gate_bwd(bf(dy), bf(h), g.act ? bf(z) : nullptr, bf(dh), ptr<const float>(w), rs, eps, g.act, rows, D, g.rows,
                             g.stride, bf_out(dx), bf_out(dres), bf_out(dz), ptr<float>(dw), ptr<void>(ws),
                             (size_t)ws.numel(), stream_of(dev)));
  const Tensor out[4] = {dx, dres, dz, dw};
  return tuple_of(out);
}

// --------------------------------------------------------------- rotary
PyObject *rope(Args &a) {
  const char *fn = "gdn_rope";
  const Tensor &q = a.tensor("q"), &k = a.maybe("k"), &pos = a.tensor("positions"), &freq = a.tensor("inv_freq");
  const int inter = a.int32("interleaved"), inverse = a.int32("inverse");
  const float f = a.real("attention_factor");
  Tensor qo = a.maybe("q_out"), ko = a.maybe("k_out");
  const auto device = on_gpu(q, "q");
  const at::Device dev = q.device();
  const int64_t ldq = token_stride(q, "q", dev), T = q.size(0), D = q.size(2);
  int64_t ldk = 0, HK = 0;
  if (k.defined()) {
    ldk = token_stride(k, "k", dev);
    HK = k.size(1);
    if (k.size(0) != T || k.size(2) != D) value_error("gdn_rope: k must have the tokens and the head size of q");
  } else if (ko.defined()) {
    value_error("gdn_rope: k_out without k");
  }
  need(pos, "positions", at::kInt, dev, 1);
  need(freq, "inv_freq", at::kFloat, dev, 1);
  if (pos.size(0) != T) value_error("gdn_rope: one position for each token is needed");
  auto out = [&](Tensor &o, const Tensor &x, const char *name) {
    if (!o.defined()) {
      o = empty(x.sizes(), at::kBFloat16, dev);
    } else {
      need(o, name, at::kBFloat16, dev, 3);
      if (o.sizes() != x.sizes()) value_error(std::string("gdn_rope: ") + name + " must have the shape " + shape_text(x));
    }
  };
  out(qo, q, "q_out");
  if (k.defined()) out(ko, k, "k_out");
  done(fn, gdn_rope(bf(q), bf(k), ptr<const int32_t>(pos), ptr<const float>(freq), T, fits32(q.size(1), "HQ"), fits32(HK, "HK"),
                    fits32(D, "D"), fits32(2 * freq.size(0), "rotary_dim"), inter, inverse, f, ldq, ldk, bf_out(qo), bf_out(ko),
                    stream_of(dev)));
  const Tensor r[2] = {qo, ko};
  return tuple_of(r);
}

// ----------------------------------------------------------- paged cache
PyObject *paged_plan(Args &a) {
  const char *fn = "gdn_paged_plan";
  const Tensor &cached = a.tensor("cached_lens"), &cu = a.tensor("cu_seqlens"), &table = a.tensor("block_table");
  const Tensor &fp = a.tensor("free_pages"), &nf = a.tensor("num_free");
  const int bs = a.int32("page_size"), T = a.int32("num_tokens");
  const Tensor &st = a.maybe("dev_status");
  const auto device = on_gpu(cached, "cached_lens");
  const at::Device dev = cached.device();
  need(cached, "cached_lens", at::kInt, dev, 1);
  need(cu, "cu_seqlens", at::kInt, dev, 1);
  need(table, "block_table", at::kInt, dev, 2);
  need(fp, "free_pages", at::kInt, dev, 1);
  need(nf, "num_free", at::kInt, dev, 1);
  if (st.defined()) need(st, "dev_status", at::kInt, dev, 1);
  const int64_t N = cached.size(0);
  if (cu.size(0) != N + 1 || table.size(0) != N || nf.size(0) != 1)
    value_error("gdn_paged_plan: cu_seqlens [N + 1], block_table [N, width] and num_free [1] must agree");
  if (T < 0) value_error("gdn_paged_plan: num_tokens must not be negative");
  const Tensor lens = empty({N}, at::kInt, dev), slots = empty({T}, at::kInt, dev), pos = empty({T}, at::kInt, dev);
  const Tensor left = empty({1}, at::kInt, dev);
  done(fn, gdn_paged_plan(ptr<const int32_t>(cached), ptr<const int32_t>(cu), fits32(N, "N"), T, ptr<int32_t>(table),
                          fits32(table.size(1), "width"), ptr<const int32_t>(fp), fits32(fp.size(0), "F"), ptr<const int32_t>(nf),
                          bs, ptr<int32_t>(lens), ptr<int32_t>(slots), ptr<int32_t>(pos), ptr<int32_t>(left), ptr<int32_t>(st),
                          stream_of(dev)));
  const Tensor r[4] = {lens, slots, pos, left};
  return tuple_of(r);
}

struct Cache {
  int P, HK, bs, D;
};
Cache cache_of(const Tensor &kc, const Tensor &vc, const Tensor &ks, const Tensor &vs, const at::Device &dev, const char *fn) {
  need(kc, "k_cache", at::kFloat8_e4m3fn, dev, 4);
  need(vc, "v_cache", at::kFloat8_e4m3fn, dev, 4);
  need(ks, "k_scale", at::kFloat, dev, 2);
  need(vs, "v_scale", at::kFloat, dev, 2);
  if (vc.sizes() != kc.sizes() || ks.size(0) != kc.size(0) || ks.size(1) != kc.size(1) || vs.sizes() != ks.sizes())
    value_error(std::string(fn) + ": caches must be [P, HK, page_size, D] and scales [P, HK]");
  return {fits32(kc.size(0), "P"), fits32(kc.size(1), "HK"), fits32(kc.size(2), "page_size"), fits32(kc.size(3), "D")};
}

PyObject *kv8_append(Args &a) {
  const char *fn = "gdn_kv8_append";
  const Tensor &k = a.tensor("k"), &v = a.tensor("v"), &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache");
  const Tensor &ks = a.tensor("k_scale"), &vs = a.tensor("v_scale"), &slots = a.tensor("slot_mapping"), &st = a.maybe("dev_status");
  const auto device = on_gpu(k, "k");
  const at::Device dev = k.device();
  const int64_t ldk = token_stride(k, "k", dev), ldv = token_stride(v, "v", dev);
  const Cache c = cache_of(kc, vc, ks, vs, dev, fn);
  need(slots, "slot_mapping", at::kInt, dev, 1);
  if (st.defined()) need(st, "dev_status", at::kInt, dev, 1);
  if (k.sizes() != v.sizes() || k.size(1) != c.HK || k.size(2) != c.D || slots.size(0) != k.size(0))
    value_error("gdn_kv8_append: k, v must be [T, HK, D] of the cache and slot_mapping [T]");
  done(fn, gdn_kv8_append(bf(k), bf(v), ldk, ldv, ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<float>(ks), ptr<float>(vs),
                          ptr<const int32_t>(slots), k.size(0), c.P, c.HK, c.D, c.bs, ptr<int32_t>(st), stream_of(dev)));
  Py_RETURN_NONE;
}

PyObject *kv8_attention(Args &a) {
  const char *fn = "gdn_kv8_attention";
  const Tensor &q = a.tensor("q"), &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache"), &ks = a.tensor("k_scale");
  const Tensor &vs = a.tensor("v_scale"), &table = a.tensor("block_table"), &lens = a.tensor("seq_lens"), &cu = a.maybe("cu_seqlens");
  const int max_q = a.int32("max_q_len");
  const long long max_seq_arg = a.integer("max_seq_len");  // -1: all places of a table row
  const float scale = a.real("scale");
  Tensor o = a.maybe("o");
  const Tensor &lse = a.maybe("lse");
  Tensor ws = a.maybe("workspace");
  const Tensor &st = a.maybe("dev_status");
  const auto device = on_gpu(q, "q");
  const at::Device dev = q.device();
  const int64_t ldq = token_stride(q, "q", dev), T = q.size(0), HQ = q.size(1), D = q.size(2);
  const Cache c = cache_of(kc, vc, ks, vs, dev, fn);
  need(table, "block_table", at::kInt, dev, 2);
  need(lens, "seq_lens", at::kInt, dev, 1);
  const int64_t N = table.size(0), width = table.size(1);
  if (c.D != D || lens.size(0) != N)
    value_error("gdn_kv8_attention: q and the caches must agree in D, block_table and seq_lens in N");
  if (cu.defined()) {
    need(cu, "cu_seqlens", at::kInt, dev, 1);
    if (cu.size(0) != N + 1) value_error("gdn_kv8_attention: cu_seqlens must be [N + 1]");
  }
  if (o.defined()) {
    need(o, "o", at::kBFloat16, dev, 3);
    if (o.sizes() != q.sizes()) value_error("gdn_kv8_attention: o must have the shape of q");
  } else {
    o = empty(q.sizes(), at::kBFloat16, dev);
  }
  if (lse.defined()) {
    need(lse, "lse", at::kFloat, dev, 2);
    if (lse.size(0) != T || lse.size(1) != HQ) value_error("gdn_kv8_attention: lse must be [T, HQ]");
  }
  if (st.defined()) need(st, "dev_status", at::kInt, dev, 1);
  const int n = fits32(N, "N"), t = fits32(T, "T"), hq = fits32(HQ, "HQ");
  const int max_seq = fits32(max_seq_arg < 0 ? width * c.bs : max_seq_arg, "max_seq_len");
  if (ws.defined()) {
    need(ws, "workspace", at::kByte, dev, 1);
  } else {
    const int64_t bytes = (int64_t)gdn_kv8_attention_workspace_size(n, t, hq, c.HK, c.D, max_q, max_seq);
    if (bytes) ws = empty({bytes}, at::kByte, dev);
  }
  done(fn, gdn_kv8_attention(bf(q), ldq, ptr<const uint8_t>(kc), ptr<const uint8_t>(vc), ptr<const float>(ks), ptr<const float>(vs),
                             ptr<const int32_t>(table), fits32(width, "width"), ptr<const int32_t>(lens), ptr<const int32_t>(cu), n,
                             t, c.P, hq, c.HK, c.D, c.bs, max_q, max_seq, scale, bf_out(o), ptr<float>(lse), ptr<void>(ws),
                             ws.defined() ? (size_t)ws.numel() : 0, ptr<int32_t>(st), stream_of(dev)));
  return wrap(o);
}

// ---------------------------------------------------- activations in 8 bits
std::vector<int64_t> scales_of(const Tensor &x) {
  std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = (shape.back() + 127) / 128;
  return shape;
}
void coded(const Tensor &codes, const Tensor &scale, const char *name, const char *scale_name, const at::Device &dev, const char *fn) {
  need(codes, name, at::kFloat8_e4m3fn, dev, -1);
  need(scale, scale_name, at::kFloat, dev, -1);
  if (codes.dim() < 1 || codes.size(-1) < 1) value_error(std::string(fn) + ": " + name + " must be [.., D], got " + shape_text(codes));
  const std::vector<int64_t> want = scales_of(codes);
  if (scale.sizes() != at::IntArrayRef(want)) value_error(std::string(fn) + ": " + scale_name + " must be [.., ceil(D / 128)]");
}
int64_t rows_in(const Tensor &x) {  // of the last dimension's size
  int64_t n = 1;
  for (int64_t i = 0; i + 1 < x.dim(); ++i) n *= x.size(i);
  return n;
}

PyObject *act8_save(Args &a) {
  const char *fn = "gdn_act8_save";
  const Tensor &x = a.tensor("x");
  Tensor codes = a.maybe("codes"), scale = a.maybe("scale");
  const auto device = on_gpu(x, "x");
  const at::Device dev = x.device();
  kind(x, "x", at::kBFloat16, dev);
  if (x.dim() < 1 || x.size(-1) < 1) value_error(std::string(fn) + ": x must be [.., D], got " + shape_text(x));
  const Gate g = rows_of(x, "x", fn);
  if (!codes.defined()) codes = empty(x.sizes(), at::kFloat8_e4m3fn, dev);
  else if (codes.sizes() != x.sizes()) value_error(std::string(fn) + ": codes must have the shape " + shape_text(x));
  if (!scale.defined()) scale = empty(scales_of(x), at::kFloat, dev);
  coded(codes, scale, "codes", "scale", dev, fn);
  done(fn, gdn_act8_save(bf(x), rows_in(x), fits32(x.size(-1), "D"), g.rows, g.stride, ptr<uint8_t>(codes), ptr<float>(scale),
                         stream_of(dev)));
  const Tensor out[2] = {codes, scale};
  return tuple_of(out);
}

PyObject *act8_load(Args &a) {
  const char *fn = "gdn_act8_load";
  const Tensor &codes = a.tensor("codes"), &scale = a.tensor("scale");
  Tensor y = a.maybe("out");
  const auto device = on_gpu(codes, "codes");
  const at::Device dev = codes.device();
  coded(codes, scale, "codes", "scale", dev, fn);
  if (y.defined()) like(y, "out", codes, fn);
  else y = empty(codes.sizes(), at::kBFloat16, dev);
  done(fn, gdn_act8_load(ptr<const uint8_t>(codes), ptr<const float>(scale), rows_in(codes), fits32(codes.size(-1), "D"), bf_out(y),
                         stream_of(dev)));
  return wrap(y);
}

PyObject *norm_gate_save8(Args &a) {
  const char *fn = "gdn_norm_gate_save8";
  const Tensor &x = a.tensor("x"), &w = a.tensor("weight"), &res = a.maybe("residual"), &z = a.maybe("z");
  const int act = a.int32("activation");
  const float eps = a.real("eps"), rs = a.real("res_scale");
  const auto device = on_gpu(x, "x");
  const at::Device dev = x.device();
  need(x, "x", at::kBFloat16, dev, -1);
  const int D = width_of(x, w, fn);
  const Gate g = gate_of(z, x, act, fn);
  if (res.defined()) like(res, "residual", x, fn);
  const std::vector<int64_t> groups = scales_of(x);
  const Tensor y = empty(x.sizes(), at::kBFloat16, dev), h = res.defined() ? empty(x.sizes(), at::kBFloat16, dev) : Tensor();
  const Tensor h8 = empty(x.sizes(), at::kFloat8_e4m3fn, dev), hs = empty(groups, at::kFloat, dev);
  const Tensor z8 = g.act ? empty(x.sizes(), at::kFloat8_e4m3fn, dev) : Tensor(), zs = g.act ? empty(groups, at::kFloat, dev) : Tensor();
  done(fn, gdn_norm_gate_save8(bf(x), bf(res), g.act ? bf(z) : nullptr, ptr<const float>(w), rs, eps, g.act, x.numel() / D, D, g.rows,
                               g.stride, bf_out(y), bf_out(h), ptr<uint8_t>(h8), ptr<float>(hs), ptr<uint8_t>(z8), ptr<float>(zs),
                               stream_of(dev)));
  const Tensor out[6] = {y, h, h8, hs, z8, zs};
  return tuple_of(out);
}

PyObject *norm_gate_bwd8(Args &a) {
  const char *fn = "gdn_norm_gate_bwd8";
  const Tensor &dy = a.tensor("dy"), &h8 = a.tensor("h_codes"), &hs = a.tensor("h_scale"), &w = a.tensor("weight");
  const Tensor &z8 = a.maybe("z_codes"), &zs = a.maybe("z_scale"), &dh = a.maybe("dh");
  const int act = a.int32("activation");
  const float eps = a.real("eps"), rs = a.real("res_scale");
  Tensor ws = a.maybe("workspace");
  const auto device = on_gpu(dy, "dy");
  const at::Device dev = dy.device();
  need(dy, "dy", at::kBFloat16, dev, -1);
  const int D = width_of(dy, w, fn);
  auto coded_like = [&](const Tensor &codes, const Tensor &scale, const char *name, const char *scale_name) {
    coded(codes, scale, name, scale_name, dev, fn);
    if (codes.sizes() != dy.sizes()) value_error(std::string(fn) + ": " + name + " must have the shape " + shape_text(dy));
  };
  coded_like(h8, hs, "h_codes", "h_scale");
  if (z8.defined() != zs.defined()) value_error(std::string(fn) + ": z_codes and z_scale belong together");
  if (z8.defined()) {
    if (act == 0) value_error(std::string(fn) + ": a gate z needs an activation");
    coded_like(z8, zs, "z_codes", "z_scale");
  }
  if (dh.defined()) like(dh, "dh", dy, fn);
  const int used = z8.defined() ? act : 0;
  const Tensor dx = empty(dy.sizes(), at::kBFloat16, dev), dw = empty(w.sizes(), at::kFloat, dev);
  const Tensor dres = dh.defined() ? empty(dy.sizes(), at::kBFloat16, dev) : Tensor();
  const Tensor dz = used ? empty(dy.sizes(), at::kBFloat16, dev) : Tensor();
  const int64_t rows = dy.numel() / D;
  if (ws.defined()) need(ws, "workspace", at::kByte, dev, 1);
  else ws = empty({(int64_t)gdn_norm_gate_bwd_workspace_size(rows, D)}, at::kByte, dev);
  done(fn, gdn_norm_gate_bwd8(bf(dy), ptr<const uint8_t>(h8), ptr<const float>(hs), ptr<const uint8_t>(z8), ptr<const float>(zs), bf(dh),
                              ptr<const float>(w), rs, eps, used, rows, D, bf_out(dx), bf_out(dres), bf_out(dz), ptr<float>(dw),
                              ptr<void>(ws), (size_t)ws.numel(), stream_of(dev)));
  const Tensor out[4] = {dx, dres, dz, dw};
  return tuple_of(out);
}

// ---------------------------------------------------- training attention
struct Attn {
  int64_t ldq, ldk, ldv;
  int N, Tq, Tk, HQ, HK, D;
};
Attn attention_of(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &cu, const Tensor &cu_k, const Tensor &st, const char *fn) {
  const at::Device dev = q.device();
  Attn s{};
  s.ldq = token_stride(q, "q", dev);
  s.ldk = token_stride(k, "k", dev);
  s.ldv = token_stride(v, "v", dev);
  if (k.sizes() != v.sizes() || k.size(2) != q.size(2))
    value_error(std::string(fn) + ": q must be [Tq, HQ, D] and k, v [Tk, HK, D]");
  int64_t N = 1;
  if (cu.defined()) {
    need(cu, "cu_seqlens", at::kInt, dev, 1);
    if (cu.size(0) < 1) value_error(std::string(fn) + ": cu_seqlens must be [N + 1]");
    N = cu.size(0) - 1;
  }
  if (cu_k.defined()) {
    need(cu_k, "cu_seqlens_k", at::kInt, dev, 1);
    if (!cu.defined() || cu_k.size(0) != N + 1) value_error(std::string(fn) + ": cu_seqlens_k must be [N + 1], as cu_seqlens");
  } else if (cu.defined() && k.size(0) != q.size(0)) {
    value_error(std::string(fn) + ": keys of other lengths than the rows' need cu_seqlens_k");
  }
  if (st.defined()) need(st, "dev_status", at::kInt, dev, 1);
  s.N = fits32(N, "N");
  s.Tq = fits32(q.size(0), "Tq");
  s.Tk = fits32(k.size(0), "Tk");
  s.HQ = fits32(q.size(1), "HQ");
  s.HK = fits32(k.size(1), "HK");
  s.D = fits32(q.size(2), "D");
  return s;
}

PyObject *attention_fwd(Args &a) {
  const char *fn = "gdn_attention_fwd";
  const Tensor &q = a.tensor("q"), &k = a.tensor("k"), &v = a.tensor("v"), &cu = a.maybe("cu_seqlens"), &cu_k = a.maybe("cu_seqlens_k");
  const int causal = a.int32("causal");
  const float scale = a.real("scale");
  Tensor o = a.maybe("o"), lse = a.maybe("lse");
  const Tensor &st = a.maybe("dev_status");
  const auto device = on_gpu(q, "q");
  const at::Device dev = q.device();
  const Attn s = attention_of(q, k, v, cu, cu_k, st, fn);
  if (o.defined()) like(o, "o", q, fn);
  else o = empty(q.sizes(), at::kBFloat16, dev);
  if (lse.defined()) {
    need(lse, "lse", at::kFloat, dev, 2);
    if (lse.size(0) != s.Tq || lse.size(1) != s.HQ) value_error("gdn_attention_fwd: lse must be [Tq, HQ]");
  } else {
    lse = empty({s.Tq, s.HQ}, at::kFloat, dev);
  }
  done(fn, gdn_attention_fwd(bf(q), s.ldq, bf(k), s.ldk, bf(v), s.ldv, ptr<const int32_t>(cu), ptr<const int32_t>(cu_k), s.N, s.Tq,
                             s.Tk, s.HQ, s.HK, s.D, causal, scale, bf_out(o), ptr<float>(lse), ptr<int32_t>(st), stream_of(dev)));
  const Tensor out[2] = {o, lse};
  return tuple_of(out);
}

PyObject *attention_bwd(Args &a) {
  const char *fn = "gdn_attention_bwd";
  const Tensor &dout = a.tensor("do"), &q = a.tensor("q"), &k = a.tensor("k"), &v = a.tensor("v"), &o = a.tensor("o"), &lse = a.tensor("lse");
  const Tensor &cu = a.maybe("cu_seqlens"), &cu_k = a.maybe("cu_seqlens_k");
  const int causal = a.int32("causal");
  const float scale = a.real("scale");
  Tensor ws = a.maybe("workspace");
  const Tensor &st = a.maybe("dev_status");
  const auto device = on_gpu(q, "q");
  const at::Device dev = q.device();
  const Attn s = attention_of(q, k, v, cu, cu_k, st, fn);
  like(dout, "do", q, fn);
  like(o, "o", q, fn);
  need(lse, "lse", at::kFloat, dev, 2);
  if (lse.size(0) != s.Tq || lse.size(1) != s.HQ) value_error("gdn_attention_bwd: lse must be [Tq, HQ]");
  const Tensor dq = empty(q.sizes(), at::kBFloat16, dev), dk = empty(k.sizes(), at::kBFloat16, dev), dv = empty(v.sizes(), at::kBFloat16, dev);
  if (ws.defined()) need(ws, "workspace", at::kByte, dev, 1);
  else ws = empty({(int64_t)gdn_attention_bwd_workspace_size(s.N, s.Tq, s.Tk, s.HQ, s.HK, s.D)}, at::kByte, dev);
  done(fn, gdn_attention_bwd(bf(dout), bf(q), s.ldq, bf(k), s.ldk, bf(v), s.ldv, bf(o), ptr<const float>(lse), ptr<const int32_t>(cu),
                             ptr<const int32_t>(cu_k), s.N, s.Tq, s.Tk, s.HQ, s.HK, s.D, causal, scale, bf_out(dq), bf_out(dk),
                             bf_out(dv), ptr<void>(ws), (size_t)ws.numel(), ptr<int32_t>(st), stream_of(dev)));
  const Tensor out[3] = {dq, dk, dv};
  return tuple_of(out);
}

PyObject *set_errors(Args &a) {  // the exceptions that this module raises beside Python's own
  for (PyObject **at : {&g_error, &g_memory_error}) {
    PyObject *o = a.next();
    Py_INCREF(o);
    Py_XDECREF(*at);
    *at = o;
  }
  Py_RETURN_NONE;
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(norm_gate),  ENTRY(norm_gate_bwd), ENTRY(rope),      ENTRY(paged_plan),
                           ENTRY(kv8_append), ENTRY(kv8_attention), ENTRY(attention_fwd), ENTRY(attention_bwd),
                           ENTRY(act8_save),  ENTRY(act8_load),  ENTRY(norm_gate_save8), ENTRY(norm_gate_bwd8),
                           ENTRY(set_errors), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_gdn_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_torch(void) { return PyModule_Create(&g_module); }
