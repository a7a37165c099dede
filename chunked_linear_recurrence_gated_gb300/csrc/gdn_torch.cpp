// Python entry of the layer operators (include/gdn_layer.h) for torch tensors:
// argument checks, output and workspace allocation, the call into the C ABI on
// the current stream of the tensors' device. Host code only. A generation step
// makes these calls once per layer and token, and on the Grace host a dozen
// tensors' attributes read from Python cost several times the launch: one step
// of one sequence takes 15.5 us of host time that way and 4.6 us this way.
#include <Python.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn_conv.h"
#include "gdn_layer.h"

namespace {

using at::Tensor;
using Sizes = std::initializer_list<int64_t>;

struct BadValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct BadType : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Refused {  // a status of the C ABI
  gdn_status status;
  const char* where;
};

PyObject* g_error = nullptr;  // GdnError(status, where)

std::string described(const Tensor& t) {
  std::ostringstream s;
  s << t.sizes() << " " << t.scalar_type() << " on " << t.device() << " with strides "
    << t.strides();
  return s.str();
}

// ------------------------------------------------------------------ arguments
const Tensor& tensor(PyObject* a, const char* name) {
  if (!THPVariable_Check(a)) throw BadType(std::string(name) + ": a tensor is expected");
  return THPVariable_Unpack(a);
}
const Tensor* optional(PyObject* a, const char* name) {
  return a == Py_None ? nullptr : &tensor(a, name);
}
float number(PyObject* a) {
  const double x = PyFloat_AsDouble(a);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}
int choice(PyObject* a) {
  const long x = PyLong_AsLong(a);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return (int)x;
}

int dtype_code(at::ScalarType t) {
  if (t == at::kFloat) return GDN_DTYPE_F32;
  if (t == at::kBFloat16) return GDN_DTYPE_BF16;
  throw BadType(std::string("unsupported dtype ") + c10::toString(t));
}

// The first tensor of a call: its GPU and number of dimensions.
int on_gpu(const char* name, const Tensor& t, int64_t ndim) {
  if (!t.is_cuda() || t.dim() != ndim)
    throw BadValue(std::string(name) + ": a CUDA tensor with " + std::to_string(ndim) +
                   " dimensions is expected, got " + described(t));
  return t.get_device();
}
void want(const char* name, const Tensor& t, at::IntArrayRef sizes, at::ScalarType type, int dev,
          bool contiguous) {
  if (t.sizes() == sizes && t.scalar_type() == type && t.is_cuda() && t.get_device() == dev &&
      (!contiguous || t.is_contiguous()))
    return;
  std::ostringstream s;
  s << name << ": expected " << (contiguous ? "contiguous " : "") << sizes << " " << type
    << " on cuda:" << dev << ", got " << described(t);
  throw BadValue(s.str());
}
void* ptr(const char* name, const Tensor& t, Sizes sizes, at::ScalarType type, int dev) {
  want(name, t, at::IntArrayRef(sizes), type, dev, true);
  return t.data_ptr();
}
void* ptr(const char* name, const Tensor* t, Sizes sizes, at::ScalarType type, int dev) {
  return t ? ptr(name, *t, sizes, type, dev) : nullptr;
}
void* like(const char* name, const Tensor* t, const Tensor& other, at::ScalarType type, int dev) {
  if (!t) return nullptr;
  want(name, *t, other.sizes(), type, dev, true);
  return t->data_ptr();
}

// Stride of the rows of t [..., n1, .., nk] (k = inner trailing dimensions that
// have to be dense) when its leading dimensions flatten to one.
long long rows(const char* name, const Tensor& t, int64_t inner) {
  const auto st = t.strides();
  const auto sh = t.sizes();
  const int64_t dim = t.dim();
  if (dim < inner) throw BadValue(std::string(name) + ": too few dimensions");
  int64_t dense = 1;
  for (int64_t i = dim - 1; i >= dim - inner; --i) {
    if (sh[i] != 1 && st[i] != dense)
      throw BadValue(std::string(name) + ": the last " + std::to_string(inner) +
                     " dimensions must be dense, got " + described(t));
    dense *= sh[i];
  }
  if (t.numel() == 0) return dense;  // no rows: the strides say nothing
  int64_t ld = dense, n = 1;
  for (int64_t i = dim - inner - 1; i >= 0; --i) {
    if (sh[i] == 1) continue;
    if (n == 1)
      ld = st[i];
    else if (st[i] != ld * n)
      throw BadValue(std::string(name) + ": the rows must have one stride, got " + described(t));
    n *= sh[i];
  }
  return ld;
}
long long rows_of(const char* name, const Tensor& t, at::IntArrayRef sizes, int64_t inner,
                  at::ScalarType type, int dev) {
  want(name, t, sizes, type, dev, false);
  return rows(name, t, inner);
}

int narrow_int(int64_t n) {  // sizes of the C ABI are int
  if (n > 0x7fffffff) throw BadValue("a dimension is past the 32-bit range");
  return (int)n;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
void check(gdn_status s, const char* where) {
  if (s != GDN_OK) throw Refused{s, where};
}
Tensor scratch(const Tensor* given, size_t bytes, const Tensor& at_device, int dev) {
  if (!given)
    return at::empty({(int64_t)std::max<size_t>(bytes, 256)},
                     at_device.options().dtype(at::kByte));
  if (!given->is_cuda() || given->get_device() != dev || !given->is_contiguous())
    throw BadValue("workspace: a contiguous CUDA tensor is expected, got " + described(*given));
  return *given;
}

struct Indices {
  const int *slot_in, *slot_out, *cu, *commit;
  int64_t N;
};
Indices indices(PyObject* const* a, int64_t n_tok, int dev) {
  const Tensor *in = optional(a[0], "slot_in"), *out = optional(a[1], "slot_out"),
               *cu = optional(a[2], "cu_seqlens"), *commit = optional(a[3], "n_commit");
  const int64_t N = cu ? cu->numel() - 1 : n_tok;
  return {(const int*)ptr("slot_in", in, {N}, at::kInt, dev),
          (const int*)ptr("slot_out", out, {N}, at::kInt, dev),
          (const int*)ptr("cu_seqlens", cu, {N + 1}, at::kInt, dev),
          (const int*)ptr("n_commit", commit, {N}, at::kInt, dev), N};
}

// ------------------------------------------------------------------ operators
// q k v g beta S slot_in slot_out cu_seqlens n_commit rate bias q_scale eps o
PyObject* step(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
               &g = tensor(a[3], "g"), &beta = tensor(a[4], "beta"), &S = tensor(a[5], "S");
  const int dev = on_gpu("q", q, 3);
  on_gpu("v", v, 3);
  on_gpu("S", S, 4);
  const auto type = q.scalar_type();
  const int64_t n = q.size(0), Hk = q.size(1), dk = q.size(2), H = v.size(1), dv = v.size(2);
  gdn_step_shape s = {};
  s.ldk = rows_of("k", k, {n, Hk, dk}, 2, type, dev);
  s.ldv = rows_of("v", v, {n, H, dv}, 2, type, dev);
  s.ldg = rows_of("g", g, {n, H}, 1, type, dev);
  s.ldb = rows_of("beta", beta, {n, H}, 1, type, dev);
  s.ldq = rows("q", q, 2);
  const Indices ix = indices(a + 6, n, dev);
  s.N = narrow_int(ix.N), s.n_tok = narrow_int(n), s.n_slots = narrow_int(S.size(0));
  s.H = narrow_int(H), s.Hk = narrow_int(Hk), s.dk = narrow_int(dk), s.dv = narrow_int(dv);
  s.dtype = dtype_code(type);
  s.q_scale = number(a[12]), s.eps = number(a[13]);
  const void* rate = ptr("rate", optional(a[10], "rate"), {H}, at::kFloat, dev);
  const void* bias = ptr("bias", optional(a[11], "bias"), {H}, at::kFloat, dev);
  void* pS = ptr("S", S, {S.size(0), H, dk, dv}, at::kFloat, dev);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  const Tensor* given = optional(a[14], "o");
  const Tensor o = given ? *given : at::empty({n, H, dv}, q.options());
  check(gdn_step(&s, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                 (const float*)rate, (const float*)bias, (float*)pS, ix.slot_in, ix.slot_out,
                 ix.cu, ix.commit, ptr("o", o, {n, H, dv}, type, dev), stream_of(dev)),
        "gdn_step");
  return THPVariable_Wrap(o);
}

// x w b state slot_in slot_out cu_seqlens n_commit act y
PyObject* conv_step(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &state = tensor(a[3], "state");
  const int dev = on_gpu("x", x, 2);
  on_gpu("w", w, 2);
  on_gpu("state", state, 3);
  const auto type = x.scalar_type();
  const int64_t n = x.size(0), C = x.size(1), W = w.size(1);
  const Indices ix = indices(a + 4, n, dev);
  gdn_conv_step_shape s = {};
  s.N = narrow_int(ix.N), s.n_tok = narrow_int(n), s.n_slots = narrow_int(state.size(0));
  s.C = narrow_int(C), s.W = narrow_int(W), s.dtype = dtype_code(type), s.act = choice(a[8]);
  s.ldx = rows("x", x, 1);
  const void* pw = ptr("w", w, {C, W}, at::kFloat, dev);
  const void* pb = ptr("b", optional(a[2], "b"), {C}, at::kFloat, dev);
  void* ps = ptr("state", state, {state.size(0), W - 1, C}, type, dev);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  const Tensor* given = optional(a[9], "y");
  const Tensor y = given ? *given : at::empty({n, C}, x.options());
  check(gdn_conv_step(&s, x.data_ptr(), (const float*)pw, (const float*)pb, ps, ix.slot_in,
                      ix.slot_out, ix.cu, ix.commit, ptr("y", y, {n, C}, type, dev),
                      stream_of(dev)),
        "gdn_conv_step");
  return THPVariable_Wrap(y);
}

struct Prep {
  gdn_prep_shape s;
  int dev;
  int64_t B, T, H, Hk, dk;
  const void *q, *k, *xg, *xb;
  const float *rate, *bias;
};
// q k xg xb rate bias, and at `last` q_scale eps
Prep prep_args(PyObject* const* a, int last) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &xg = tensor(a[2], "xg"),
               &xb = tensor(a[3], "xb");
  Prep p = {};
  p.dev = on_gpu("q", q, 4);
  on_gpu("xg", xg, 3);
  const auto type = q.scalar_type();
  p.B = q.size(0), p.T = q.size(1), p.Hk = q.size(2), p.dk = q.size(3), p.H = xg.size(2);
  p.s.ldk = rows_of("k", k, q.sizes(), 2, type, p.dev);
  p.s.ldg = rows_of("xg", xg, {p.B, p.T, p.H}, 1, type, p.dev);
  p.s.ldb = rows_of("xb", xb, {p.B, p.T, p.H}, 1, type, p.dev);
  p.s.ldq = rows("q", q, 2);
  p.s.rows = narrow_int(p.B * p.T), p.s.H = narrow_int(p.H), p.s.Hk = narrow_int(p.Hk);
  p.s.dk = narrow_int(p.dk), p.s.dtype = dtype_code(type);
  p.s.q_scale = number(a[last]), p.s.eps = number(a[last + 1]);
  p.q = q.data_ptr(), p.k = k.data_ptr(), p.xg = xg.data_ptr(), p.xb = xb.data_ptr();
  p.rate = (const float*)ptr("rate", tensor(a[4], "rate"), {p.H}, at::kFloat, p.dev);
  p.bias = (const float*)ptr("bias", tensor(a[5], "bias"), {p.H}, at::kFloat, p.dev);
  return p;
}

PyObject* tuple_of(std::initializer_list<const Tensor*> ts) {
  PyObject* t = PyTuple_New((Py_ssize_t)ts.size());
  if (!t) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* x : ts) {
    PyObject* o = x && x->defined() ? THPVariable_Wrap(*x) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(t);
      throw python_error();
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// q k xg xb rate bias q_scale eps
PyObject* prep_fwd(PyObject* const* a) {
  const Prep p = prep_args(a, 6);
  const auto opt = tensor(a[0], "q").options();
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  const Tensor qn = at::empty({p.B, p.T, p.H, p.dk}, opt), kn = at::empty(qn.sizes(), opt),
               g = at::empty({p.B, p.T, p.H}, opt), beta = at::empty(g.sizes(), opt);
  check(gdn_prep_fwd(&p.s, p.q, p.k, p.xg, p.xb, p.rate, p.bias, qn.data_ptr(), kn.data_ptr(),
                     g.data_ptr(), beta.data_ptr(), stream_of(p.dev)),
        "gdn_prep_fwd");
  return tuple_of({&qn, &kn, &g, &beta});
}

// q k xg xb rate bias dq dk dg dbeta q_scale eps workspace
PyObject* prep_bwd(PyObject* const* a) {
  const Prep p = prep_args(a, 10);
  const Tensor& q = tensor(a[0], "q");
  const auto type = q.scalar_type();
  const Sizes heads = {p.B, p.T, p.H, p.dk}, gates = {p.B, p.T, p.H};
  const void* dqn = ptr("dq", tensor(a[6], "dq"), heads, type, p.dev);
  const void* dkn = ptr("dk", tensor(a[7], "dk"), heads, type, p.dev);
  const void* dg = ptr("dg", tensor(a[8], "dg"), gates, type, p.dev);
  const void* db = ptr("dbeta", tensor(a[9], "dbeta"), gates, type, p.dev);
  const auto opt = q.options(), fopt = opt.dtype(at::kFloat);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  const Tensor ws = scratch(optional(a[12], "workspace"), gdn_prep_workspace_bytes(&p.s), q, p.dev);
  const Tensor oq = at::empty(q.sizes(), opt), ok = at::empty(q.sizes(), opt),
               og = at::empty(at::IntArrayRef(gates), opt), ob = at::empty(og.sizes(), opt),
               drate = at::empty({p.H}, fopt), dbias = at::empty({p.H}, fopt);
  check(gdn_prep_bwd(&p.s, p.q, p.k, p.xg, p.xb, p.rate, p.bias, dqn, dkn, dg, db, oq.data_ptr(),
                     ok.data_ptr(), og.data_ptr(), ob.data_ptr(), (float*)drate.data_ptr(),
                     (float*)dbias.data_ptr(), ws.data_ptr(), ws.nbytes(), stream_of(p.dev)),
        "gdn_prep_bwd");
  return tuple_of({&oq, &ok, &og, &ob, &drate, &dbias});
}

struct Gate {
  gdn_gate_norm_shape s;
  int dev;
  const void *o, *z;
  const float* w;
};
// o z w act, and at `eps` eps
Gate gate_args(PyObject* const* a, int act, int eps) {
  const Tensor &o = tensor(a[0], "o"), &z = tensor(a[1], "z"), &w = tensor(a[2], "w");
  Gate p = {};
  p.dev = on_gpu("o", o, 4);
  const auto type = o.scalar_type();
  p.s.rows = narrow_int(o.size(0) * o.size(1)), p.s.H = narrow_int(o.size(2));
  p.s.d = narrow_int(o.size(3)), p.s.dtype = dtype_code(type), p.s.act = choice(a[act]);
  p.s.ldz = rows_of("z", z, o.sizes(), 2, type, p.dev);
  p.s.eps = number(a[eps]);
  want("o", o, o.sizes(), type, p.dev, true);
  p.o = o.data_ptr(), p.z = z.data_ptr();
  p.w = (const float*)ptr("w", w, {o.size(3)}, at::kFloat, p.dev);
  return p;
}

// o z w act eps y
PyObject* gate_norm_fwd(PyObject* const* a) {
  const Gate p = gate_args(a, 3, 4);
  const Tensor &o = tensor(a[0], "o"), *given = optional(a[5], "y");
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  const Tensor y = given ? *given : at::empty(o.sizes(), o.options());
  check(gdn_gate_norm_fwd(&p.s, p.o, p.z, p.w, like("y", &y, o, o.scalar_type(), p.dev),
                          stream_of(p.dev)),
        "gdn_gate_norm_fwd");
  return THPVariable_Wrap(y);
}

// o z w dy act eps workspace
PyObject* gate_norm_bwd(PyObject* const* a) {
  const Gate p = gate_args(a, 4, 5);
  const Tensor &o = tensor(a[0], "o"), &w = tensor(a[2], "w"), &dy = tensor(a[3], "dy");
  const void* pdy = like("dy", &dy, o, o.scalar_type(), p.dev);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  const Tensor ws =
      scratch(optional(a[6], "workspace"), gdn_gate_norm_workspace_bytes(&p.s), o, p.dev);
  const Tensor dout = at::empty(o.sizes(), o.options()), dz = at::empty(o.sizes(), o.options()),
               dw = at::empty(w.sizes(), w.options());
  check(gdn_gate_norm_bwd(&p.s, p.o, p.z, p.w, pdy, dout.data_ptr(), dz.data_ptr(),
                          (float*)dw.data_ptr(), ws.data_ptr(), ws.nbytes(), stream_of(p.dev)),
        "gdn_gate_norm_bwd");
  return tuple_of({&dout, &dz, &dw});
}

struct Res {
  gdn_res_norm_shape s;
  int dev;
  const float *w, *w_post, *scale;
};
// h, w, w_post, scale, eps; type: of x and y
Res res_args(const char* name, const Tensor& h, at::ScalarType type, PyObject* w, PyObject* w_post,
             PyObject* scale, PyObject* eps) {
  if (!h.is_cuda() || h.dim() < 1)
    throw BadValue(std::string(name) + ": a CUDA tensor is expected, got " + described(h));
  Res p = {};
  p.dev = h.get_device();
  const int64_t C = h.size(-1);
  p.s.rows = narrow_int(h.numel() / std::max<int64_t>(C, 1)), p.s.C = narrow_int(C);
  p.s.dtype = dtype_code(type), p.s.res_dtype = dtype_code(h.scalar_type());
  p.s.eps = number(eps);
  want(name, h, h.sizes(), h.scalar_type(), p.dev, true);
  p.w = (const float*)ptr("w", tensor(w, "w"), {C}, at::kFloat, p.dev);
  p.w_post = (const float*)ptr("w_post", optional(w_post, "w_post"), {C}, at::kFloat, p.dev);
  p.scale = (const float*)ptr("scale", optional(scale, "scale"), {C}, at::kFloat, p.dev);
  return p;
}

// h x w w_post scale eps h_out y bf16 (without x and y: whether y is bf16, None: h's dtype)
PyObject* res_norm_fwd(PyObject* const* a) {
  const Tensor &h = tensor(a[0], "h"), *x = optional(a[1], "x"), *ho = optional(a[6], "h_out"),
               *yo = optional(a[7], "y");
  const auto type = x               ? x->scalar_type()
                    : yo            ? yo->scalar_type()
                    : a[8] == Py_None ? h.scalar_type()
                    : choice(a[8])  ? at::kBFloat16
                                    : at::kFloat;
  if ((x || yo) && a[8] != Py_None && (choice(a[8]) != 0) != (type == at::kBFloat16))
    throw BadValue(std::string("dtype: ") + (x ? "x" : "y") + " is " + c10::toString(type));
  const Res p = res_args("h", h, type, a[2], a[3], a[4], a[5]);
  const void* px = like("x", x, h, type, p.dev);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  const Tensor y = yo ? *yo : at::empty(h.sizes(), h.options().dtype(type));
  const Tensor out = ho ? *ho : x ? at::empty(h.sizes(), h.options()) : Tensor();
  check(gdn_res_norm_fwd(&p.s, h.data_ptr(), px, p.w, p.w_post, p.scale,
                         like("h_out", out.defined() ? &out : nullptr, h, h.scalar_type(), p.dev),
                         like("y", &y, h, type, p.dev), stream_of(p.dev)),
        "gdn_res_norm_fwd");
  return tuple_of({&out, &y});
}

// h_out x w dy dh_out w_post scale eps dh workspace
PyObject* res_norm_bwd(PyObject* const* a) {
  const Tensor &h = tensor(a[0], "h_out"), *x = optional(a[1], "x"), &w = tensor(a[2], "w"),
               &dy = tensor(a[3], "dy"), *dho = optional(a[4], "dh_out"),
               *dho2 = optional(a[8], "dh");
  const auto type = dy.scalar_type(), rtype = h.scalar_type();
  const Res p = res_args("h_out", h, type, a[2], a[5], a[6], a[7]);
  const void* px = like("x", x, h, type, p.dev);
  const void* pdy = like("dy", &dy, h, type, p.dev);
  const void* pdho = like("dh_out", dho, h, rtype, p.dev);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  const Tensor ws =
      scratch(optional(a[9], "workspace"), gdn_res_norm_workspace_bytes(&p.s), h, p.dev);
  const Tensor dh = dho2 ? *dho2 : at::empty(h.sizes(), h.options());
  const bool same = !p.w_post && !p.scale && (type == rtype || !x);
  const Tensor dx = same ? dh : at::empty(h.sizes(), dy.options());
  const Tensor dw = at::empty(w.sizes(), w.options());
  const Tensor dpost = p.w_post ? at::empty(w.sizes(), w.options()) : Tensor();
  const Tensor dscale = p.scale ? at::empty(w.sizes(), w.options()) : Tensor();
  check(gdn_res_norm_bwd(&p.s, h.data_ptr(), px, p.w, p.w_post, p.scale, pdy, pdho,
                         like("dh", &dh, h, rtype, p.dev), same ? nullptr : dx.data_ptr(),
                         (float*)dw.data_ptr(), p.w_post ? (float*)dpost.data_ptr() : nullptr,
                         p.scale ? (float*)dscale.data_ptr() : nullptr, ws.data_ptr(),
                         ws.nbytes(), stream_of(p.dev)),
        "gdn_res_norm_bwd");
  return tuple_of({&dh, &dx, &dw, &dpost, &dscale});
}

// name t inner
PyObject* row_stride(PyObject* const* a) {
  const char* name = PyUnicode_AsUTF8(a[0]);
  if (!name) throw python_error();
  return PyLong_FromLongLong(rows(name, tensor(a[1], name), choice(a[2])));
}

// ---------------------------------------------------------------------- module
template <PyObject* (*F)(PyObject* const*), int NARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != NARGS) {
    PyErr_Format(PyExc_TypeError, "%d arguments are expected, got %zd", NARGS, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const BadType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const Refused& r) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", (int)r.status, r.where) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s: status %d", r.where, (int)r.status);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(type);
  Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, (PyCFunction)(void*)(entry<f, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(step, 15),
                         ENTRY(conv_step, 10),
                         ENTRY(prep_fwd, 8),
                         ENTRY(prep_bwd, 13),
                         ENTRY(gate_norm_fwd, 6),
                         ENTRY(gate_norm_bwd, 7),
                         ENTRY(res_norm_fwd, 9),
                         ENTRY(res_norm_bwd, 10),
                         ENTRY(row_stride, 3),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_torch() { return PyModule_Create(&module); }
