// Arguments of the calls whose work on the device is often shorter than a Python
// binding's: torch tensors checked, outputs allocated, C descriptors filled, and the
// call of the C ABI made, on the stream that the caller names.  No arithmetic.
// binding.py holds the public functions, their defaults and documentation; a wrong
// argument raises ValueError here, the library's own code is returned to it.
// (In Python the checks and descriptors of one token's head norms took 24 us, those
// of AdamW over 122 tensors 185.)
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>

#include <cmath>
#include <cstring>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/muonclip.h"

namespace {

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Raised {};                        // Python's own error is set
[[noreturn]] void bad(const std::string& what) { throw Bad(what); }

// The positional arguments of a call, taken in order.
struct Args {
  PyObject* const* at;
  Py_ssize_t left;
  PyObject* next() {
    if (left-- <= 0) bad("too few arguments");
    return *at++;
  }
  // an optional tensor: undefined for None
  at::Tensor maybe(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return {};
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  at::Tensor tensor(const char* name) {
    at::Tensor t = maybe(name);
    if (!t.defined()) bad(std::string(name) + " must be a tensor");
    return t;
  }
  int64_t number(const char* name, int64_t none) {
    PyObject* o = next();
    if (o == Py_None) return none;
    if (!PyLong_Check(o)) bad(std::string(name) + " must be an integer");
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    return x;
  }
  double real() {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return x;
  }
  int64_t whole() {
    const long long x = PyLong_AsLongLong(next());
    if (x == -1 && PyErr_Occurred()) throw Raised();
    return x;
  }
  mc_stream_t stream() {
    const unsigned long long x = PyLong_AsUnsignedLongLong(next());
    if (PyErr_Occurred()) throw Raised();
    return reinterpret_cast<mc_stream_t>(static_cast<uintptr_t>(x));
  }
};

std::string shape_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}
int32_t dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MC_F32;
    case at::kBFloat16: return MC_BF16;
    case at::kFloat8_e4m3fn: return MC_F8E4M3;
    default: return -1;
  }
}
// Every given tensor on the first one's CUDA device.
void one_device(const at::Tensor& first, std::initializer_list<const at::Tensor*> others) {
  if (!first.is_cuda()) bad("expected CUDA tensors");
  for (const at::Tensor* t : others)
    if (t->defined() && (!t->is_cuda() || t->get_device() != first.get_device())) bad("every tensor must be on one device");
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
at::Tensor fresh(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) { return at::empty(shape, like.options().dtype(type)); }

// A given tensor of this shape and type, contiguous, or a new one.
void whole_tensor(const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type) {
  if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous())
    bad(std::string(name) + " must be a contiguous " + shape_of(shape) + " tensor of " + toString(type));
}
at::Tensor whole_or_new(const char* name, const at::Tensor& t, const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  if (!t.defined()) return fresh(like, shape, type);
  whole_tensor(name, t, shape, type);
  return t;
}
// A [tokens, heads, features] operand of this shape and type.
void rows(const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type) {
  if (t.sizes() != shape || t.scalar_type() != type) bad(std::string(name) + " must be " + shape_of(shape) + " of " + toString(type));
  if (t.stride(2) != 1 && shape[2] > 1) bad(std::string(name) + ": expected unit stride along the features");
}
// A given output like `like`, or a new one, its rows padded to a multiple of `per`
// features (which the attention calls' strides must be).
at::Tensor rows_or_new(const char* name, const at::Tensor& t, const at::Tensor& like, at::IntArrayRef shape, int64_t per = 1) {
  if (t.defined()) {
    rows(name, t, shape, like.scalar_type());
    return t;
  }
  if (shape[2] % per == 0) return fresh(like, shape, like.scalar_type());
  return fresh(like, {shape[0], shape[1], (shape[2] + per - 1) / per * per}, like.scalar_type()).narrow(2, 0, shape[2]);
}
int64_t workspace_bytes(const at::Tensor& t) {
  if (!t.is_contiguous()) bad("workspace must be contiguous");
  return t.numel() * t.element_size();
}
void check_status(const at::Tensor& t) {
  if (t.defined() && (t.scalar_type() != at::kInt || t.numel() < 1)) bad("status must be an int32 tensor");
}
PyObject* object(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// The C call with other Python threads running.
template <typename F>
int called(F f) {
  int code;
  Py_BEGIN_ALLOW_THREADS
  code = f();
  Py_END_ALLOW_THREADS
  return code;
}

// ------------------------------------------------------------------ head norms
struct Heads {
  mc_heads h;
  std::vector<int64_t> q, k;
  at::ScalarType type;
};
Heads heads_of(const at::Tensor& q, const at::Tensor& k, const at::Tensor& positions, double theta, int64_t rot, double eps) {
  Heads r;
  if (q.dim() != 3 || (dtype_of(q) != MC_F32 && dtype_of(q) != MC_BF16)) bad("q: expected [T, heads, d] of bfloat16 or float32");
  r.type = q.scalar_type();
  r.q = q.sizes().vec();
  r.k = {r.q[0], 0, r.q[2]};
  if (k.defined()) {
    if (k.dim() != 3 || k.size(0) != r.q[0] || k.size(2) != r.q[2] || k.scalar_type() != r.type)
      bad("keys must be [" + std::to_string(r.q[0]) + ", heads, " + std::to_string(r.q[2]) + "] of q's type");
    r.k[1] = k.size(1);
    if (r.k[1] == 0) bad("keys without a head: pass none");
  }
  if (positions.defined()) whole_tensor("positions", positions, {r.q[0]}, at::kInt);
  if (r.q[1] > INT32_MAX || r.k[1] > INT32_MAX || r.q[2] > INT32_MAX || rot > INT32_MAX || rot < INT32_MIN) bad("sizes are too large");
  memset(&r.h, 0, sizeof r.h);
  r.h.T = r.q[0];
  r.h.heads_q = (int32_t)r.q[1];
  r.h.heads_k = (int32_t)r.k[1];
  r.h.d = (int32_t)r.q[2];
  r.h.rot = (int32_t)rot;
  r.h.dtype = dtype_of(q);
  r.h.eps = (float)eps;
  r.h.theta = theta;
  r.h.positions = static_cast<const int32_t*>(ptr(positions));
  return r;
}
struct View {
  void* p;
  int64_t token, head;
};
View view(const at::Tensor& t) { return t.defined() ? View{t.data_ptr(), t.stride(0), t.stride(1)} : View{nullptr, 0, 0}; }

PyObject* norm_rope(Args a) {
  const at::Tensor q = a.tensor("q"), k = a.maybe("k"), wq = a.maybe("wq"), wk = a.maybe("wk"), positions = a.maybe("positions");
  const double theta = a.real();
  const int64_t rot = a.number("rot", q.dim() ? q.sizes().back() : 0);
  const double eps = a.real();
  at::Tensor out_q = a.maybe("out_q"), out_k = a.maybe("out_k"), rstd = a.maybe("rstd");
  const bool norm = a.whole() != 0;
  const mc_stream_t stream = a.stream();
  one_device(q, {&k, &wq, &wk, &positions, &out_q, &out_k, &rstd});
  Heads s = heads_of(q, k, positions, theta, rot, eps);
  s.h.no_norm = !norm;
  if (!norm && rstd.defined()) bad("rstd goes with a norm");
  rows("q", q, s.q, s.type);
  if (k.defined()) rows("k", k, s.k, s.type);
  else if (wk.defined() || out_k.defined()) bad("wk and out_k go with k");
  if (wq.defined()) whole_tensor("wq", wq, {s.q[2]}, s.type);
  if (wk.defined()) whole_tensor("wk", wk, {s.q[2]}, s.type);
  out_q = rows_or_new("out_q", out_q, q, s.q);
  if (k.defined()) out_k = rows_or_new("out_k", out_k, k, s.k);
  if (norm) rstd = whole_or_new("rstd", rstd, q, {s.q[0], s.q[1] + s.k[1]}, at::kFloat);
  const View x = view(q), y = view(k), xo = view(out_q), yo = view(out_k);
  const int code = called([&] {
    return mc_head_norm_rope(&s.h, x.p, x.token, x.head, y.p, y.token, y.head, ptr(wq), ptr(wk), xo.p, xo.token, xo.head, yo.p, yo.token,
                             yo.head, static_cast<float*>(ptr(rstd)), stream);
  });
  return Py_BuildValue("iNNN", code, object(out_q), object(out_k), object(rstd));
}

PyObject* norm_rope_backward(Args a) {
  const at::Tensor dyq = a.tensor("dyq"), dyk = a.maybe("dyk"), q = a.tensor("q"), k = a.maybe("k"), rstd = a.maybe("rstd"), wq = a.maybe("wq"),
                   wk = a.maybe("wk"), positions = a.maybe("positions");
  const double theta = a.real();
  const int64_t rot = a.number("rot", q.dim() ? q.sizes().back() : 0);
  at::Tensor dq = a.maybe("dq"), dk = a.maybe("dk"), dwq = a.maybe("dwq"), dwk = a.maybe("dwk"), ws = a.maybe("workspace");
  const bool norm = a.whole() != 0;
  const mc_stream_t stream = a.stream();
  one_device(q, {&dyq, &dyk, &k, &rstd, &wq, &wk, &positions, &dq, &dk, &dwq, &dwk, &ws});
  Heads s = heads_of(q, k, positions, theta, rot, 0.0);
  s.h.no_norm = !norm;
  if (norm != rstd.defined()) bad(norm ? "rstd must be a tensor" : "rstd goes with a norm");
  if (k.defined() != dyk.defined() || (!k.defined() && (wk.defined() || dk.defined() || dwk.defined())))
    bad("k, dyk, wk, dk and dwk go together");
  rows("q", q, s.q, s.type);
  rows("dyq", dyq, s.q, s.type);
  if (rstd.defined()) whole_tensor("rstd", rstd, {s.q[0], s.q[1] + s.k[1]}, at::kFloat);
  dq = rows_or_new("dq", dq, q, s.q);
  if (k.defined()) {
    rows("k", k, s.k, s.type);
    rows("dyk", dyk, s.k, s.type);
    dk = rows_or_new("dk", dk, k, s.k);
  }
  const int64_t d = s.q[2];
  if (wq.defined()) whole_tensor("wq", wq, {d}, s.type);
  if (wk.defined()) whole_tensor("wk", wk, {d}, s.type);
  if (wq.defined() || dwq.defined()) dwq = whole_or_new("dwq", dwq, q, {d}, at::kFloat);
  if (wk.defined() || dwk.defined()) dwk = whole_or_new("dwk", dwk, q, {d}, at::kFloat);
  size_t bytes = 0;
  if (dwq.defined() || dwk.defined()) {
    if (ws.defined()) {
      bytes = (size_t)workspace_bytes(ws);
    } else {
      const int code = mc_head_norm_rope_backward_workspace_size((int32_t)d, &bytes);
      if (code) return Py_BuildValue("iOOOO", code, Py_None, Py_None, Py_None, Py_None);
      ws = fresh(q, {(int64_t)bytes}, at::kByte);
    }
  }
  const View g = view(dyq), gk = view(dyk), x = view(q), y = view(k), o = view(dq), ok = view(dk);
  const int code = called([&] {
    return mc_head_norm_rope_backward(&s.h, g.p, g.token, g.head, gk.p, gk.token, gk.head, x.p, x.token, x.head, y.p, y.token, y.head,
                                      static_cast<const float*>(ptr(rstd)), ptr(wq), ptr(wk), o.p, o.token, o.head, ok.p, ok.token, ok.head,
                                      static_cast<float*>(ptr(dwq)), static_cast<float*>(ptr(dwk)), ptr(ws), bytes, stream);
  });
  return Py_BuildValue("iNNNN", code, object(dq), object(dk), object(dwq), object(dwk));
}

// ------------------------------------------------------------ packed attention
mc_packed_desc packed_desc(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& offsets, PyObject* scale) {
  if (q.dim() != 3 || k.dim() != 3 || v.dim() != 3) bad("q, k and v must be [T, heads, features]");
  if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || v.size(0) != q.size(0) || v.size(1) != k.size(1))
    bad("k must be [T, H_kv, d] and v [T, H_kv, d_v] with q's tokens and width");
  const int32_t type = dtype_of(q);
  if ((type != MC_F32 && type != MC_BF16) || k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
    bad("q, k and v must share a supported dtype");
  if (q.stride(2) != 1 || k.stride(2) != 1 || v.stride(2) != 1) bad("feature axes must be contiguous");
  if (offsets.dim() != 1 || offsets.scalar_type() != at::kInt || !offsets.is_contiguous() || offsets.numel() < 2)
    bad("offsets must be a contiguous int32 tensor of one value more than there are sequences");
  for (const int64_t n : {q.size(0), q.size(1), q.size(2), k.size(1), v.size(2), offsets.numel()})
    if (n > INT32_MAX) bad("sizes are too large");
  mc_packed_desc d;
  memset(&d, 0, sizeof d);
  d.T = (int32_t)q.size(0);
  d.nseq = (int32_t)offsets.numel() - 1;
  d.H = (int32_t)q.size(1);
  d.H_kv = (int32_t)k.size(1);
  d.d = (int32_t)q.size(2);
  d.d_v = (int32_t)v.size(2);
  d.dtype = type;
  if (scale == Py_None) {
    d.scale = (float)(1.0 / std::sqrt((double)q.size(2)));
  } else {
    const double x = PyFloat_AsDouble(scale);            // beyond fp32: inf, which the library refuses
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    d.scale = (float)x;
  }
  d.offsets = static_cast<const int32_t*>(ptr(offsets));
  d.q = ptr(q);
  d.k = ptr(k);
  d.v = ptr(v);
  for (int i = 0; i < 2; ++i) {
    d.q_strides[i] = q.stride(i);
    d.k_strides[i] = k.stride(i);
    d.v_strides[i] = v.stride(i);
  }
  return d;
}
// The workspace's bytes; a new one where none is given.  A code of the library, or 0.
int packed_workspace(const mc_packed_desc& d, bool backward, const at::Tensor& like, at::Tensor& ws, size_t& bytes) {
  if (ws.defined()) {
    bytes = (size_t)workspace_bytes(ws);
    return 0;
  }
  const int code = qk_attention_packed_workspace_size(&d, backward, &bytes);
  if (!code) ws = fresh(like, {(int64_t)bytes}, at::kByte);
  return code;
}

PyObject* packed_size(Args a) {
  const at::Tensor q = a.tensor("q"), k = a.tensor("k"), v = a.tensor("v"), offsets = a.tensor("offsets");
  const mc_packed_desc d = packed_desc(q, k, v, offsets, Py_None);
  size_t bytes = 0;
  const int code = qk_attention_packed_workspace_size(&d, a.whole() != 0, &bytes);
  return Py_BuildValue("iK", code, (unsigned long long)bytes);
}

PyObject* packed_forward(Args a) {
  const at::Tensor q = a.tensor("q"), k = a.tensor("k"), v = a.tensor("v"), offsets = a.tensor("offsets");
  PyObject* scale = a.next();
  at::Tensor out = a.maybe("out");
  PyObject* lse_arg = a.next();
  at::Tensor lse;
  if (lse_arg != Py_None && lse_arg != Py_True && lse_arg != Py_False) {
    if (!THPVariable_Check(lse_arg)) bad("lse must be a tensor, or True for a new one");
    lse = THPVariable_Unpack(lse_arg);
  }
  at::Tensor smax = a.maybe("smax");
  const bool accumulate = a.whole() != 0;
  at::Tensor ws = a.maybe("workspace"), status = a.maybe("status");
  const mc_stream_t stream = a.stream();
  one_device(q, {&k, &v, &offsets, &out, &lse, &smax, &ws, &status});
  mc_packed_desc d = packed_desc(q, k, v, offsets, scale);
  d.fill = (out.defined() ? 0 : MC_FILL_O) | (lse.defined() ? 0 : MC_FILL_LSE);        // of new ones every row is written
  out = rows_or_new("out", out, q, {q.size(0), q.size(1), v.size(2)}, 8);
  if (lse.defined() || lse_arg == Py_True) lse = whole_or_new("lse", lse, q, {q.size(1), q.size(0)}, at::kFloat);
  if (!smax.defined() && accumulate) bad("accumulate goes with a smax to combine");
  smax = whole_or_new("smax", smax, q, {q.size(1)}, at::kFloat);
  check_status(status);
  size_t bytes = 0;
  int code = packed_workspace(d, false, q, ws, bytes);
  const int64_t st[2] = {out.stride(0), out.stride(1)};
  if (!code)
    code = called([&] {
      return qk_attention_packed_forward(&d, ptr(out), st, static_cast<float*>(ptr(lse)), static_cast<float*>(ptr(smax)), accumulate, ptr(ws),
                                         bytes, static_cast<int32_t*>(ptr(status)), stream);
    });
  return Py_BuildValue("iNNN", code, object(out), object(lse), object(smax));
}

PyObject* packed_backward(Args a) {
  const at::Tensor q = a.tensor("q"), k = a.tensor("k"), v = a.tensor("v"), out = a.tensor("out"), lse = a.tensor("lse"), dout = a.tensor("dout"),
                   offsets = a.tensor("offsets");
  PyObject* scale = a.next();
  at::Tensor dq = a.maybe("dq"), dk = a.maybe("dk"), dv = a.maybe("dv"), ws = a.maybe("workspace"), status = a.maybe("status");
  const mc_stream_t stream = a.stream();
  one_device(q, {&k, &v, &out, &lse, &dout, &offsets, &dq, &dk, &dv, &ws, &status});
  mc_packed_desc d = packed_desc(q, k, v, offsets, scale);
  d.fill = (dq.defined() ? 0 : MC_FILL_DQ) | (dk.defined() ? 0 : MC_FILL_DK) | (dv.defined() ? 0 : MC_FILL_DV);
  const int64_t shape[3] = {q.size(0), q.size(1), v.size(2)};
  rows("out", out, shape, q.scalar_type());
  rows("dout", dout, shape, q.scalar_type());
  whole_tensor("lse", lse, {q.size(1), q.size(0)}, at::kFloat);
  dq = rows_or_new("dq", dq, q, q.sizes(), 8);
  dk = rows_or_new("dk", dk, k, k.sizes(), 8);
  dv = rows_or_new("dv", dv, v, v.sizes(), 8);
  check_status(status);
  size_t bytes = 0;
  int code = packed_workspace(d, true, q, ws, bytes);
  mc_packed_grad g;
  memset(&g, 0, sizeof g);
  g.o = ptr(out);
  g.lse = static_cast<const float*>(ptr(lse));
  g.d_o = ptr(dout);
  g.dq = ptr(dq);
  g.dk = ptr(dk);
  g.dv = ptr(dv);
  for (int i = 0; i < 2; ++i) {
    g.o_strides[i] = out.stride(i);
    g.do_strides[i] = dout.stride(i);
    g.dq_strides[i] = dq.stride(i);
    g.dk_strides[i] = dk.stride(i);
    g.dv_strides[i] = dv.stride(i);
  }
  if (!code) code = called([&] { return qk_attention_packed_backward(&d, &g, ptr(ws), bytes, static_cast<int32_t*>(ptr(status)), stream); });
  return Py_BuildValue("iNNN", code, object(dq), object(dk), object(dv));
}

// ----------------------------------------------------------------------- AdamW
// A list or tuple of tensors.
struct Tensors {
  PyObject* list = nullptr;
  Py_ssize_t n = 0;
  Tensors(PyObject* o, const char* name) {
    if (o == Py_None) return;
    if (!PyList_Check(o) && !PyTuple_Check(o)) bad(std::string(name) + " must be a list of tensors");
    list = o;
    n = PySequence_Fast_GET_SIZE(o);
    for (Py_ssize_t i = 0; i < n; ++i)
      if (!THPVariable_Check(PySequence_Fast_GET_ITEM(o, i))) bad(std::string(name) + " must be a list of tensors");
  }
  const at::Tensor& operator[](Py_ssize_t i) const { return THPVariable_Unpack(PySequence_Fast_GET_ITEM(list, i)); }
};

PyObject* adamw(Args a) {
  const Tensors P(a.next(), "P"), G(a.next(), "G"), M(a.next(), "M"), V(a.next(), "V"), ms(a.next(), "m_scales"), vs(a.next(), "v_scales");
  mc_adamw_hparams hp;
  memset(&hp, 0, sizeof hp);
  hp.lr = a.real();
  hp.beta1 = a.real();
  hp.beta2 = a.real();
  hp.eps = a.real();
  hp.weight_decay = a.real();
  PyObject* step = a.next();
  const at::Tensor grad_scale = a.maybe("grad_scale"), status = a.maybe("status");
  const mc_stream_t stream = a.stream();
  at::Tensor counted;
  if (THPVariable_Check(step)) {
    counted = THPVariable_Unpack(step);
    if (counted.numel() != 1 || counted.scalar_type() != at::kLong) bad("step must be an integer or one int64 value on the device");
    hp.step_device = static_cast<const int64_t*>(counted.data_ptr());
  } else {
    hp.step = PyLong_AsLongLong(step);
    if (hp.step == -1 && PyErr_Occurred()) throw Raised();
  }
  const Py_ssize_t n = P.n;
  if (G.n != n || M.n != n || V.n != n) bad("P, G, M and V must have one length");
  const bool eight = ms.list != nullptr;
  if (eight != (vs.list != nullptr)) bad("m_scales and v_scales go together");
  if (eight && (ms.n != n || vs.n != n)) bad("m_scales and v_scales must have P's length");
  if (n > INT32_MAX) bad("too many tensors");
  int device = -1;
  auto here = [&](const at::Tensor& t) {
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device)) bad("every tensor must be on one CUDA device");
    device = (int)t.get_device();
  };
  auto plain = [&](const at::Tensor& t) {
    here(t);
    if (!t.is_contiguous()) bad("every tensor must be contiguous");
    return t.data_ptr();
  };
  std::vector<mc_adamw_tensor> ts((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    mc_adamw_tensor& t = ts[(size_t)i];
    memset(&t, 0, sizeof t);
    t.p = plain(P[i]);
    t.g = plain(G[i]);
    t.m = plain(M[i]);
    t.v = plain(V[i]);
    t.n = P[i].numel();
    if (G[i].numel() != t.n || M[i].numel() != t.n || V[i].numel() != t.n) bad("P, G, M and V must agree in size, tensor by tensor");
    t.p_dtype = dtype_of(P[i]);
    t.g_dtype = dtype_of(G[i]);
    t.state_dtype = dtype_of(M[i]);
    if ((t.p_dtype != MC_F32 && t.p_dtype != MC_BF16) || (t.g_dtype != MC_F32 && t.g_dtype != MC_BF16)) bad("P and G must be bfloat16 or float32");
    if (t.state_dtype != (eight ? MC_F8E4M3 : MC_F32) || dtype_of(V[i]) != t.state_dtype)
      bad("M and V must be float32, or float8_e4m3fn with m_scales and v_scales");
    if (eight) {
      t.m_scale = static_cast<float*>(plain(ms[i]));
      t.v_scale = static_cast<float*>(plain(vs[i]));
      const int64_t blocks = (t.n + MC_ADAMW_BLOCK - 1) / MC_ADAMW_BLOCK;
      if (ms[i].numel() != blocks || vs[i].numel() != blocks || dtype_of(ms[i]) != MC_F32 || dtype_of(vs[i]) != MC_F32)
        bad("scales must be float32, one per 128 values of their tensor");
    }
  }
  for (const at::Tensor* t : std::initializer_list<const at::Tensor*>{&grad_scale, &status, &counted})
    if (t->defined()) here(*t);
  if (grad_scale.defined() && (grad_scale.numel() != 1 || grad_scale.scalar_type() != at::kFloat)) bad("grad_scale must be one float32 value");
  check_status(status);
  const int code = called([&] {
    return mc_adamw_step(ts.data(), (int32_t)n, &hp, static_cast<const float*>(ptr(grad_scale)), static_cast<int32_t*>(ptr(status)), stream);
  });
  return Py_BuildValue("(i)", code);
}

// torch's errors become the Python exceptions that they are elsewhere (an allocation that fails:
// torch.cuda.OutOfMemoryError).
template <PyObject* (*F)(Args)>
PyObject* entry(PyObject*, PyObject* const* at, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  try {
    return F(Args{at, count});
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(norm_rope),      ENTRY(norm_rope_backward), ENTRY(packed_size), ENTRY(packed_forward),
                         ENTRY(packed_backward), ENTRY(adamw),              {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host(void) { return PyModule_Create(&module); }
