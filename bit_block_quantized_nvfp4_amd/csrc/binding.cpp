// Python entry points of the token sort, block norm and e4m3 operators: tensors
// in, checks, outputs where none are given, one call of the C ABI on torch's
// current stream, tensors out.  No arithmetic.  ops.py documents the arguments
// and passes them on by position; doing the marshalling here instead of there
// takes a call's host time from 8 or more to 4 us, which is most of a decode
// step's call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "../../include/moe_nvfp4.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Shape = at::IntArrayRef;

PyObject* g_moe_error = nullptr;     // _lib.MoeError
PyObject* g_memory_error = nullptr;  // torch.OutOfMemoryError

struct Refusal {  // becomes a ValueError
  std::string text;
};
struct Raised {};  // a Python error is already set

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refusal{s.str()};
}

const char* type_name(ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

std::string shape_text(Shape s) {
  std::ostringstream o;
  o << '(';
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

// The arguments of one call, taken by position.
struct Args {
  PyObject* const* v;
  Py_ssize_t n, at = 0;
  PyObject* next() {
    if (at >= n) refuse("too few arguments");
    return v[at++];
  }
  const Tensor* maybe(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
    return &THPVariable_Unpack(o);
  }
  const Tensor& tensor(const char* name) {
    const Tensor* t = maybe(name);
    if (!t) refuse(name, " is missing");
    return *t;
  }
  int integer(const char* name) {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(name, " is out of range: ", v);
    return (int)v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw Raised{};
    return v != 0;
  }
  float number() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
  }
};

// t's device.  A call makes it the current one while it lasts (OnDevice): outputs
// and kernels go there, to that device's current stream.
c10::Device device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, " must be a device tensor");
  return t.device();
}
using OnDevice = c10::DeviceGuard;

int dtype_of(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DT_BF16;
    case at::kHalf: return MOE_DT_F16;
    case at::kFloat: return MOE_DT_F32;
    default: refuse(name, " must be bfloat16, float16 or float32, got ", type_name(t.scalar_type()));
  }
}

void two_dims(const Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(name, " must have two dimensions");
}

void* need(const Tensor& t, ScalarType type, Shape shape, c10::Device dev, const char* name) {
  if (t.device() != dev) refuse(name, " must be on ", dev.str(), ", got ", t.device().str());
  if (t.scalar_type() != type)
    refuse(name, " must be ", type_name(type), ", got ", type_name(t.scalar_type()));
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
  if (t.sizes() != shape)
    refuse(name, " must have shape ", shape_text(shape), ", got ", shape_text(t.sizes()));
  return t.data_ptr();
}

// A new tensor, as torch.empty makes it: dispatch modes see it, and torch fills it
// where deterministic algorithms ask for that.
Tensor fresh(ScalarType type, Shape shape, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// An output: the one given, checked, or a new one.
Tensor output(const Tensor* t, ScalarType type, Shape shape, c10::Device dev, const char* name) {
  if (!t) return fresh(type, shape, dev);
  need(*t, type, shape, dev, name);
  return *t;
}

Tensor scratch(const Tensor* t, size_t bytes, c10::Device dev) {
  if (!t) return fresh(at::kByte, {(int64_t)bytes}, dev);
  if (t->device() != dev || !t->is_contiguous() || (size_t)t->nbytes() < bytes)
    refuse("workspace of ", bytes, " contiguous bytes on ", dev.str(), " needed");
  return *t;
}

// Tokens of a permutation with K routed slots (and a shared one) each.  None is
// for the library to refuse, as every size is.
int tokens(const Tensor& slot_pos, int K, bool shared) {
  const int64_t per = (int64_t)K + shared, n = slot_pos.numel();
  if (K < 1 || n % per)
    refuse("slot_pos has ", n, " entries, not a multiple of ", per, " slots a token");
  if (n / per > INT32_MAX) refuse("slot_pos is too long");
  return (int)(n / per);
}

int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(name, " is too large");
  return (int)v;
}

void* stream() { return (void*)c10::hip::getCurrentHIPStream().stream(); }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// One call of the C ABI, without the interpreter's lock: a launch may have to wait
// (a full queue, the first call's kernel lookup), and other Python threads go on
// meanwhile, as they do through ctypes.  The caller's frame holds the arguments.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
int call(F f, A... a) {
  const Unlocked meanwhile;
  return f(a...);
}

void check(int status) {
  if (status >= 0) return;
  PyObject* e = PyObject_CallFunction(g_moe_error, "is", status, moe_last_error());
  if (e) {
    PyErr_SetObject(g_moe_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* wrap_all(std::initializer_list<Tensor> list) {
  PyObject* r = PyTuple_New((Py_ssize_t)list.size());
  Py_ssize_t i = 0;
  for (const Tensor& t : list) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

PyObject* dispatch(Args a) {
  const Tensor& x = a.tensor("x");
  const Tensor& pos = a.tensor("slot_pos");
  const int K = a.integer("K");
  const bool sh = a.truth();
  const Tensor* given = a.maybe("xs");
  const c10::Device dev = device_of(x, "x");
  const OnDevice on(dev);
  const int dt = dtype_of(x, "x"), T = tokens(pos, K, sh);
  two_dims(x, "x");
  const int64_t H = x.size(1), S = (int64_t)T * (K + sh);
  need(x, x.scalar_type(), {T, H}, dev, "x");
  need(pos, at::kInt, {S}, dev, "slot_pos");
  Tensor xs = output(given, x.scalar_type(), {S, H}, dev, "xs");
  check(call(moe_dispatch, x.data_ptr(), pos.data_ptr<int32_t>(), T, K, size32(H, "H"), sh, dt,
                     xs.data_ptr(), stream()));
  return wrap(xs);
}

PyObject* dispatch_grad(Args a) {
  const Tensor& dxs = a.tensor("dxs");
  const Tensor& pos = a.tensor("slot_pos");
  const int K = a.integer("K");
  const bool sh = a.truth();
  const Tensor* given = a.maybe("dx");
  const c10::Device dev = device_of(dxs, "dxs");
  const OnDevice on(dev);
  const int dt = dtype_of(dxs, "dxs"), T = tokens(pos, K, sh);
  two_dims(dxs, "dxs");
  const int64_t H = dxs.size(1), S = (int64_t)T * (K + sh);
  need(dxs, dxs.scalar_type(), {S, H}, dev, "dxs");
  need(pos, at::kInt, {S}, dev, "slot_pos");
  Tensor dx = output(given, dxs.scalar_type(), {T, H}, dev, "dx");
  check(call(moe_dispatch_grad, dxs.data_ptr(), pos.data_ptr<int32_t>(), T, K, size32(H, "H"), sh, dt,
                          dx.data_ptr(), stream()));
  return wrap(dx);
}

PyObject* combine(Args a) {
  const Tensor& y = a.tensor("y_slots");
  const Tensor& w = a.tensor("w");
  const Tensor& pos = a.tensor("slot_pos");
  const Tensor* gate = a.maybe("gate");
  const int K = a.integer("K");
  const bool sh = a.truth();
  const Tensor* given = a.maybe("out");
  const c10::Device dev = device_of(y, "y_slots");
  const OnDevice on(dev);
  const int dt = dtype_of(y, "y_slots"), T = tokens(pos, K, sh);
  two_dims(y, "y_slots");
  const int64_t H = y.size(1), S = (int64_t)T * (K + sh);
  // a longer buffer of rows may serve fewer tokens
  if (y.size(0) < S) refuse("y_slots must have ", S, " rows at least, got ", y.size(0));
  need(y, y.scalar_type(), y.sizes(), dev, "y_slots");
  const float* wp = (const float*)need(w, at::kFloat, {T, K}, dev, "w");
  const int32_t* pp = (const int32_t*)need(pos, at::kInt, {S}, dev, "slot_pos");
  const float* gp = gate ? (const float*)need(*gate, at::kFloat, {T}, dev, "gate") : nullptr;
  Tensor out = output(given, y.scalar_type(), {T, H}, dev, "out");
  const int h = size32(H, "H");
  if (dt != MOE_DT_BF16)
    check(call(moe_combine_typed, y.data_ptr(), wp, pp, gp, T, K, h, sh, dt, out.data_ptr(), stream()));
  else if (gp)
    check(call(moe_combine_gated, (const uint16_t*)y.data_ptr(), wp, pp, gp, T, K, h,
                            (uint16_t*)out.data_ptr(), stream()));
  else
    check(call(moe_combine, (const uint16_t*)y.data_ptr(), wp, pp, T, K, h, sh,
                      (uint16_t*)out.data_ptr(), stream()));
  return wrap(out);
}

PyObject* combine_grad(Args a) {
  const Tensor& dout = a.tensor("dout");
  const Tensor& y = a.tensor("y_slots");
  const Tensor& w = a.tensor("w");
  const Tensor& pos = a.tensor("slot_pos");
  const int K = a.integer("K");
  const bool sh = a.truth();
  const Tensor* gate = a.maybe("gate");
  const Tensor* dy_given = a.maybe("dy_slots");
  const Tensor* dw_given = a.maybe("dw");
  const Tensor* dgate_given = a.maybe("dgate");
  const c10::Device dev = device_of(dout, "dout");
  const OnDevice on(dev);
  const int dt = dtype_of(dout, "dout"), T = tokens(pos, K, sh);
  two_dims(dout, "dout");
  const ScalarType type = dout.scalar_type();
  const int64_t H = dout.size(1), S = (int64_t)T * (K + sh);
  need(dout, type, {T, H}, dev, "dout");
  need(y, type, {S, H}, dev, "y_slots");
  need(w, at::kFloat, {T, K}, dev, "w");
  need(pos, at::kInt, {S}, dev, "slot_pos");
  Tensor dgate;
  if (gate) {
    need(*gate, at::kFloat, {T}, dev, "gate");
    dgate = output(dgate_given, at::kFloat, {T}, dev, "dgate");
  } else if (dgate_given) {
    refuse("dgate is given without a gate");
  }
  Tensor dy = output(dy_given, type, {S, H}, dev, "dy_slots");
  Tensor dw = output(dw_given, at::kFloat, {T, K}, dev, "dw");
  check(call(moe_combine_grad, dout.data_ptr(), y.data_ptr(), w.data_ptr<float>(),
                         pos.data_ptr<int32_t>(), (const float*)ptr(gate), T, K, size32(H, "H"),
                         sh, dt, dy.data_ptr(), dw.data_ptr<float>(),
                         gate ? dgate.data_ptr<float>() : nullptr, stream()));
  return wrap_all({dy, dw, dgate});
}

PyObject* route_topk_grad(Args a) {
  const Tensor& ids = a.tensor("ids");
  const Tensor& w = a.tensor("w");
  const Tensor& dw = a.tensor("dw");
  const int E = a.integer("E");
  const Tensor* given = a.maybe("dlogits");
  const c10::Device dev = device_of(ids, "ids");
  const OnDevice on(dev);
  two_dims(ids, "ids");
  const int T = size32(ids.size(0), "T"), K = size32(ids.size(1), "K");
  if (E < 1) refuse("E must be positive");
  need(ids, at::kInt, {T, K}, dev, "ids");
  need(w, at::kFloat, {T, K}, dev, "w");
  need(dw, at::kFloat, {T, K}, dev, "dw");
  Tensor dz = output(given, at::kFloat, {T, E}, dev, "dlogits");
  check(call(moe_route_topk_grad, ids.data_ptr<int32_t>(), w.data_ptr<float>(), dw.data_ptr<float>(), T,
                            E, K, dz.data_ptr<float>(), stream()));
  return wrap(dz);
}

// The kind of a gate beside rows of this shape and type.
int gate_kind(const Tensor* gate, const Tensor& rows, c10::Device dev) {
  if (!gate) return MOE_GATE_NONE;
  if (gate->dim() == 1) {
    need(*gate, at::kFloat, {rows.size(0)}, dev, "gate");
    return MOE_GATE_TOKEN;
  }
  need(*gate, rows.scalar_type(), rows.sizes(), dev, "gate");
  return MOE_GATE_ELEMENT;
}

PyObject* block_norm(Args a) {
  const Tensor& res = a.tensor("residual");
  const Tensor* y = a.maybe("y");
  const Tensor* gate = a.maybe("gate");
  const Tensor* w_post = a.maybe("w_post");
  const Tensor* w_pre = a.maybe("w_pre");
  const float res_scale = a.number(), out_scale = a.number(), eps = a.number();
  const Tensor* r_given = a.maybe("r_out");
  const Tensor* n_given = a.maybe("n_out");
  const Tensor* sp_given = a.maybe("rstd_post");
  const Tensor* sn_given = a.maybe("rstd_pre");
  const c10::Device dev = device_of(res, "residual");
  const OnDevice on(dev);
  const int dt = dtype_of(res, "residual");
  const ScalarType type = res.scalar_type();
  two_dims(res, "residual");
  const Shape shape = res.sizes();
  const int T = size32(shape[0], "T"), H = size32(shape[1], "H");
  need(res, type, shape, dev, "residual");
  if (!y && (gate || w_post || r_given || !w_pre))
    refuse("without y only w_pre and n_out are given");
  const int kind = gate_kind(gate, res, dev);
  Tensor r, n, sp, sn;
  if (y) {
    need(*y, type, shape, dev, "y");
    r = output(r_given, type, shape, dev, "r_out");
  }
  if (w_post) {
    need(*w_post, at::kFloat, {H}, dev, "w_post");
    sp = output(sp_given, at::kFloat, {T}, dev, "rstd_post");
  } else if (sp_given) {
    refuse("rstd_post is given without w_post");
  }
  if (w_pre) {
    need(*w_pre, at::kFloat, {H}, dev, "w_pre");
    n = output(n_given, type, shape, dev, "n_out");
    sn = output(sn_given, at::kFloat, {T}, dev, "rstd_pre");
  } else if (n_given || sn_given) {
    refuse("n_out or rstd_pre is given without w_pre");
  }
  check(call(moe_block_norm, res.data_ptr(), ptr(y), ptr(gate), kind, (const float*)ptr(w_post),
                       (const float*)ptr(w_pre), res_scale, out_scale, eps, T, H, dt,
                       y ? r.data_ptr() : nullptr, w_pre ? n.data_ptr() : nullptr,
                       w_post ? sp.data_ptr<float>() : nullptr,
                       w_pre ? sn.data_ptr<float>() : nullptr, stream()));
  return wrap_all({y ? r : res, n, sp, sn});
}

PyObject* block_norm_grad(Args a) {
  const Tensor* dr = a.maybe("dr");
  const Tensor* dn = a.maybe("dn");
  const Tensor& r = a.tensor("r");
  const Tensor* y = a.maybe("y");
  const Tensor* gate = a.maybe("gate");
  const Tensor* w_post = a.maybe("w_post");
  const Tensor* w_pre = a.maybe("w_pre");
  const Tensor* sp = a.maybe("rstd_post");
  const Tensor* sn = a.maybe("rstd_pre");
  const float res_scale = a.number(), out_scale = a.number();
  const Tensor* ws_given = a.maybe("ws");
  const c10::Device dev = device_of(r, "r");
  const OnDevice on(dev);
  const int dt = dtype_of(r, "r");
  const ScalarType type = r.scalar_type();
  two_dims(r, "r");
  const Shape shape = r.sizes();
  const int T = size32(shape[0], "T"), H = size32(shape[1], "H");
  need(r, type, shape, dev, "r");
  if (!dr && !dn) refuse("dr and dn are both missing");
  if (dr) need(*dr, type, shape, dev, "dr");
  if ((dn != nullptr) != (w_pre != nullptr)) refuse("dn and w_pre are given together");
  if (!y && (gate || w_post)) refuse("a gate or w_post is given without y");
  const int kind = gate_kind(gate, r, dev);
  Tensor dres, dy, dgate, dw_post, dw_pre;
  if (w_pre) {
    need(*dn, type, shape, dev, "dn");
    need(*w_pre, at::kFloat, {H}, dev, "w_pre");
    if (!sn) refuse("w_pre needs rstd_pre");
    need(*sn, at::kFloat, {T}, dev, "rstd_pre");
    dw_pre = output(nullptr, at::kFloat, {H}, dev, "dw_pre");
  } else {
    sn = nullptr;
  }
  if (y) {
    need(*y, type, shape, dev, "y");
    dy = output(nullptr, type, shape, dev, "dy");
    if (gate) dgate = output(nullptr, gate->scalar_type(), gate->sizes(), dev, "dgate");
  }
  if (w_post) {
    need(*w_post, at::kFloat, {H}, dev, "w_post");
    if (!sp) refuse("w_post needs rstd_post");
    need(*sp, at::kFloat, {T}, dev, "rstd_post");
    dw_post = output(nullptr, at::kFloat, {H}, dev, "dw_post");
  } else {
    sp = nullptr;
  }
  dres = output(nullptr, type, shape, dev, "dresidual");
  const size_t bytes = moe_block_norm_workspace_bytes(T, H, dt);
  Tensor ws = scratch(ws_given, bytes, dev);
  check(call(
      moe_block_norm_grad,
      ptr(dr), ptr(dn), r.data_ptr(), ptr(y), ptr(gate), kind, (const float*)ptr(w_post),
      (const float*)ptr(w_pre), (const float*)ptr(sp), (const float*)ptr(sn), res_scale, out_scale,
      T, H, dt, dres.data_ptr(), y ? dy.data_ptr() : nullptr, gate ? dgate.data_ptr() : nullptr,
      w_post ? dw_post.data_ptr<float>() : nullptr, w_pre ? dw_pre.data_ptr<float>() : nullptr,
      ws.data_ptr(), bytes, stream()));
  return wrap_all({dres, dy, dgate, dw_post, dw_pre});
}

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// e4m3 codes, as such or as their bytes.
const uint8_t* codes_of(const Tensor& t, Shape shape, c10::Device dev, const char* name) {
  return (const uint8_t*)need(
      t, t.scalar_type() == at::kFloat8_e4m3fn ? at::kFloat8_e4m3fn : at::kByte, shape, dev, name);
}

PyObject* fp8_quant(Args a) {
  const Tensor& x = a.tensor("x");
  const Tensor* codes_given = a.maybe("codes");
  const Tensor* scales_given = a.maybe("scales");
  const c10::Device dev = device_of(x, "x");
  const OnDevice on(dev);
  const int dt = dtype_of(x, "x");
  two_dims(x, "x");
  const int T = size32(x.size(0), "T"), K = size32(x.size(1), "K");
  need(x, x.scalar_type(), {T, K}, dev, "x");
  Tensor codes = output(codes_given, at::kFloat8_e4m3fn, {T, K}, dev, "codes");
  Tensor scales = output(scales_given, at::kFloat, {T, blocks128(K)}, dev, "scales");
  check(call(moe_fp8_quant, x.data_ptr(), T, K, dt, (uint8_t*)codes.data_ptr(),
                      scales.data_ptr<float>(), stream()));
  return wrap_all({codes, scales});
}

PyObject* fp8_linear(Args a) {
  const Tensor& codes = a.tensor("codes");
  const Tensor& scales = a.tensor("scales");
  const Tensor& x = a.tensor("x");
  const Tensor* ws_given = a.maybe("ws");
  const Tensor* given = a.maybe("out");
  const c10::Device dev = device_of(x, "x");
  const OnDevice on(dev);
  const int dt = dtype_of(x, "x");
  two_dims(codes, "codes");
  const int N = size32(codes.size(0), "N"), K = size32(codes.size(1), "K");
  moe_fp8_matrix M;
  M.codes = codes_of(codes, {N, K}, dev, "codes");
  M.scales = (const float*)need(scales, at::kFloat, {blocks128(N), blocks128(K)}, dev, "scales");
  M.N = N;
  M.K = K;
  if (x.dim() != 2 || x.size(1) != K)
    refuse("x must be [T, ", K, "], got ", shape_text(x.sizes()));
  const int T = size32(x.size(0), "T");
  need(x, x.scalar_type(), {T, K}, dev, "x");
  Tensor out = output(given, x.scalar_type(), {T, N}, dev, "out");
  const size_t bytes = moe_fp8_linear_workspace_bytes(T, N, K);
  Tensor ws;
  if (bytes) ws = scratch(ws_given, bytes, dev);
  check(call(moe_fp8_linear, &M, x.data_ptr(), T, dt, out.data_ptr(), bytes ? ws.data_ptr() : nullptr,
                       bytes, stream()));
  return wrap(out);
}

PyObject* fp8_expert_ffn(Args a) {
  const Tensor& gu = a.tensor("gu_codes");
  const Tensor& gus = a.tensor("gu_scales");
  const Tensor& dn = a.tensor("dn_codes");
  const Tensor& dns = a.tensor("dn_scales");
  const int E = a.integer("E"), H = a.integer("H"), I = a.integer("I");
  const bool sh = a.truth();
  const Tensor& x = a.tensor("x");
  const int K = a.integer("K");
  const Tensor& offsets = a.tensor("offsets");
  const Tensor& slots = a.tensor("sorted_slot");
  const Tensor& groups = a.tensor("groups");
  const Tensor* ws_given = a.maybe("ws");
  const Tensor* given = a.maybe("y_slots");
  const c10::Device dev = device_of(x, "x");
  const OnDevice on(dev);
  if (x.dim() != 2 || x.size(1) != H) refuse("x width does not match the weight bank");
  const int T = size32(x.size(0), "T");
  if (E < 1 || I < 1 || K < 1) refuse("E, I and K must be positive");
  const int64_t G = (int64_t)E + sh, S = (int64_t)T * (K + sh);
  need(x, at::kBFloat16, {T, H}, dev, "x");
  need(offsets, at::kInt, {G + 1}, dev, "offsets");
  need(slots, at::kInt, {S}, dev, "sorted_slot");
  need(groups, at::kInt, {G + 1}, dev, "groups");
  moe_fp8_weights W;
  W.gu_codes = codes_of(gu, {G, 2 * (int64_t)I, H}, dev, "gu_codes");
  W.gu_scales = (const float*)need(gus, at::kFloat, {G, 2 * (int64_t)I / 128, H / 128}, dev, "gu_scales");
  W.dn_codes = codes_of(dn, {G, H, I}, dev, "dn_codes");
  W.dn_scales = (const float*)need(dns, at::kFloat, {G, H / 128, I / 128}, dev, "dn_scales");
  W.E = E;
  W.H = H;
  W.I = I;
  W.has_shared = sh;
  Tensor y = output(given, at::kBFloat16, {S, H}, dev, "y_slots");
  const size_t bytes = moe_fp8_expert_ffn_workspace_bytes(T, K, H, I, sh);
  Tensor ws = scratch(ws_given, bytes, dev);
  check(call(moe_fp8_expert_ffn, &W, (const uint16_t*)x.data_ptr(), T, K, offsets.data_ptr<int32_t>(),
                           slots.data_ptr<int32_t>(), groups.data_ptr<int32_t>(),
                           (uint16_t*)y.data_ptr(), ws.data_ptr(), bytes, stream()));
  return wrap(y);
}

// C++ errors end here: none passes into the interpreter.
template <PyObject* (*F)(Args)>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    return F(Args{v, n});
  } catch (const Raised&) {
  } catch (const Refusal& r) {
    PyErr_SetString(PyExc_ValueError, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory_error, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* set_errors(PyObject*, PyObject* args) {
  PyObject *moe, *memory;
  if (!PyArg_ParseTuple(args, "OO", &moe, &memory)) return nullptr;
  Py_INCREF(moe);
  Py_INCREF(memory);
  Py_XDECREF(g_moe_error);
  Py_XDECREF(g_memory_error);
  g_moe_error = moe;
  g_memory_error = memory;
  Py_RETURN_NONE;
}

#define ENTRY(f) {#f, (PyCFunction)(void (*)(void)) & entry<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ENTRY(dispatch),        ENTRY(dispatch_grad), ENTRY(combine),
    ENTRY(combine_grad),    ENTRY(route_topk_grad), ENTRY(block_norm),
    ENTRY(block_norm_grad), ENTRY(fp8_quant),     ENTRY(fp8_linear),
    ENTRY(fp8_expert_ffn),  {"set_errors", set_errors, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
