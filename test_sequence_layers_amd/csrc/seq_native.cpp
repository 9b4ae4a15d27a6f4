// The marshalling of seq.py as a CPython extension: tensors in, the C ABI of include/ttt_seq.h called on the
// current stream, tensors out. The binding is the only layer that sees the tensors' shapes: each is checked
// against the layout that the C ABI assumes before anything is called. Argument marshalling only.
//
// Why not ctypes, as for the layers themselves: a call on a few tokens takes 3 to 5 us on the device, and the
// host is what it waits for. A launch takes 3.1 us of that; from Python, the checks of a tensor took 0.4 us
// each and an output's allocation 1.2 us.
//
// A function returns its outputs, or the C ABI's status as an int where that is not TTT_OK. Wrong tensors raise
// TypeError or ValueError.
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/Allocator.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "../../include/ttt_seq.h"

namespace {

using at::Tensor;

// The library's entry points, looked up in the handle that Python has loaded.
struct Api {
#define TTT_FN(name) decltype(&::name) name
  TTT_FN(ttt_forward_layernorm);
  TTT_FN(ttt_backward_layernorm);
  TTT_FN(ttt_backward_layernorm_workspace);
  TTT_FN(ttt_forward_conv1d);
  TTT_FN(ttt_step_conv1d);
  TTT_FN(ttt_backward_conv1d);
  TTT_FN(ttt_backward_conv1d_workspace);
  TTT_FN(ttt_forward_selective_scan);
  TTT_FN(ttt_forward_selective_scan_workspace);
  TTT_FN(ttt_step_selective_scan);
  TTT_FN(ttt_backward_selective_scan);
  TTT_FN(ttt_backward_selective_scan_workspace);
#undef TTT_FN
} api;

std::string text(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

const Tensor& tensor_of(const char* name, PyObject* o) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a CUDA (HIP) tensor");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_TYPE(t.is_cuda(), name, " must be a CUDA (HIP) tensor");
  return t;
}
const Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor_of(name, o); }

// Other Python threads run while this one allocates or waits for a place in a stream's queue.
struct NoGil {
  PyThreadState* const state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

template <class F, class... A>
ttt_status enqueue(F* f, A... a) {
  const NoGil free;
  return f(a...);
}

// A tensor of the caller's that a call has written counts as changed: autograd refuses a gradient that needs its old
// values. (Tensors made in inference mode have no count.)
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// An output: the caller's tensor or a new one.
struct Out {
  Tensor t;
  PyObject* given = nullptr;
  void* p = nullptr;
  PyObject* object() const {  // a new reference, of an output that has been written
    if (!p) Py_RETURN_NONE;
    if (given) return written(THPVariable_Unpack(given)), Py_INCREF(given), given;
    return THPVariable_Wrap(t);
  }
};

struct Rows {
  const void* p = nullptr;
  long long stride = 0;
};

// The device, dtype and stream of one call, and the checks of its tensors against them.
class Call {
 public:
  Call(const char* name, const Tensor& x) : device_(x.device()), io_(x.scalar_type()), guard_(x.device()) {
    TORCH_CHECK_TYPE(io_ == at::kBFloat16 || io_ == at::kFloat, "unsupported I/O dtype ", io_, " of ", name);
    dt = io_ == at::kBFloat16 ? TTT_BF16 : TTT_F32;
    stream = c10::hip::getCurrentHIPStream(device_.index()).stream();
  }

  void* need(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype) const {
    same(name, t, shape, dtype);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.data_ptr();
  }
  void* io(const char* name, const Tensor& t, at::IntArrayRef shape) const { return need(name, t, shape, io_); }
  const float* f32(const char* name, const Tensor& t, at::IntArrayRef shape) const {
    return static_cast<const float*>(need(name, t, shape, at::kFloat));
  }
  // The same of tensors that may be left out.
  void* io(const char* name, const Tensor* t, at::IntArrayRef shape) const { return t ? io(name, *t, shape) : nullptr; }
  const float* f32(const char* name, const Tensor* t, at::IntArrayRef shape) const {
    return t ? f32(name, *t, shape) : nullptr;
  }
  const int* lengths(const Tensor* t, int64_t B) const {
    return t ? static_cast<const int*>(need("lengths", *t, {B}, at::kInt)) : nullptr;
  }

  // An activation whose last dims (`width` elements) are contiguous and whose leading dims are one run of
  // evenly spaced rows.
  Rows rows(const char* name, const Tensor& t, at::IntArrayRef shape, int64_t width) const {
    same(name, t, shape, io_);
    if (t.is_contiguous()) return {t.data_ptr(), width};
    const auto sizes = t.sizes(), strides = t.strides();
    int d = (int)sizes.size();
    for (int64_t inner = 1; inner < width;) {  // the dims that make up a row
      --d;
      TORCH_CHECK_VALUE(sizes[d] == 1 || strides[d] == inner, "the last ", width, " elements of each row of ", name,
                        " must be contiguous");
      inner *= sizes[d];
    }
    int64_t step = -1, span = 0;
    for (int i = d - 1; i >= 0; --i) {
      if (sizes[i] == 1) continue;
      if (step < 0) step = strides[i];
      else TORCH_CHECK_VALUE(strides[i] == span, "the rows of ", name, " must be evenly spaced over its leading dims");
      span = strides[i] * sizes[i];
    }
    if (step < 0) step = width;
    TORCH_CHECK_VALUE(step >= width, "the rows of ", name, " overlap");
    return {t.data_ptr(), step};
  }

  // An output of `like`'s shape and dtype. (From the allocator directly, as the workspace is: through the
  // dispatcher it takes longer.)
  Out out(const char* name, PyObject* given, const Tensor& like) const {
    Out o;
    if (given != Py_None) {
      const Tensor& t = tensor_of(name, given);
      o.p = need(name, t, like.sizes(), like.scalar_type());
      o.given = given;
    } else {
      const NoGil free;
      o.t = at::detail::empty_cuda(like.sizes(), like.scalar_type(), device_, c10::nullopt);
      o.p = o.t.data_ptr();
    }
    return o;
  }
  // The gradient of an input, none where that is not there.
  Out grad(const char* name, PyObject* given, const Tensor* of) const {
    if (of) return out(name, given, *of);
    TORCH_CHECK_VALUE(given == Py_None, name, " is given without its input");
    return Out{};
  }

  // Pointer and bytes; `held` keeps a new one until the call is enqueued (its memory is given back in the order
  // of the stream).
  void* workspace(PyObject* given, size_t need, size_t& bytes, c10::DataPtr& held) const {
    bytes = 0;
    if (given != Py_None) {
      TORCH_CHECK_VALUE(THPVariable_Check(given) && THPVariable_Unpack(given).device() == device_ &&
                            THPVariable_Unpack(given).is_contiguous(),
                        "workspace must be a contiguous tensor on ", device_);
      const Tensor& t = THPVariable_Unpack(given);
      bytes = (size_t)t.numel() * t.element_size();
      return t.data_ptr();
    }
    if (need == 0) return nullptr;
    const NoGil free;
    held = c10::GetAllocator(c10::DeviceType::CUDA)->allocate(need);
    bytes = need;
    return held.get();
  }

  ttt_dtype dt;
  hipStream_t stream;

 private:
  void same(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype) const {
    TORCH_CHECK_VALUE(t.device() == device_, name, " is on ", t.device(), ", not ", device_);
    TORCH_CHECK_VALUE(t.scalar_type() == dtype, name, " must have dtype ", dtype, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(!t.is_neg(), name, " is a negated view: resolve_neg() it first");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", text(shape), ", not ", text(t.sizes()));
  }
  const at::Device device_;
  const at::ScalarType io_;
  const c10::DeviceGuard guard_;
  const at::AutoDispatchBelowADInplaceOrView below_;  // (outputs are new memory: autograd has no part in them)
};

// Sizes go to the C ABI as int: one that does not fit is refused here.
int as_int(const char* name, int64_t v) {
  TORCH_CHECK_VALUE(v >= 0 && v <= 0x7fffffff, name, " is too large: ", v);
  return (int)v;
}
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
PyObject* status(ttt_status st) { return PyLong_FromLong(st); }

template <size_t N>
PyObject* tuple_of(const Out (&outs)[N]) {
  PyObject* r = PyTuple_New(N);
  if (!r) throw python_error();
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, outs[i].object());
  return r;
}

#define TTT_ARGS(n)                                                                        \
  if (count != n) {                                                                        \
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", n, count);           \
    return nullptr;                                                                        \
  }

// ---- layer norm -------------------------------------------------------------------------------
struct Norm {
  int M, H, D;
};
// weight [D] norms x's rows, weight [H, D] each head's D of [..., H, D].
Norm norm_of(const Tensor& x, const Tensor& weight) {
  const auto ws = weight.sizes();
  const size_t nd = ws.size();
  TORCH_CHECK_VALUE(nd == 1 || nd == 2, "weight must be [D] or [H, D]");
  TORCH_CHECK_VALUE((size_t)x.dim() > nd && x.sizes().slice(x.dim() - nd) == ws, "x must be [...", nd == 2 ? ", H" : "",
                    ", D] for a weight of ", text(ws), ", not ", text(x.sizes()));
  const int64_t H = nd == 1 ? 1 : ws[0], D = ws[nd - 1], per = H * D;
  return {as_int("x", per ? x.numel() / per : 0), as_int("weight", H), as_int("weight", D)};
}

// (x, weight, bias, eps, y)
PyObject* layernorm_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(5)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]);
  const Tensor* b = maybe("bias", a[2]);
  const Call c("x", x);
  const Norm n = norm_of(x, w);
  const Rows px = c.rows("x", x, x.sizes(), (int64_t)n.H * n.D);
  const float *pw = c.f32("weight", w, w.sizes()), *pb = c.f32("bias", b, w.sizes());
  const Out y = c.out("y", a[4], x);
  const float eps = number(a[3]);
  const ttt_status st = enqueue(api.ttt_forward_layernorm, c.dt, n.M, n.H, n.D, eps, px.p, px.stride, pw, pb, y.p,
                                c.stream);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (x, weight, d_y, eps, d_x, d_weight, d_bias, workspace)
PyObject* layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(8)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]), &dy = tensor_of("d_y", a[2]);
  const Call c("x", x);
  const Norm n = norm_of(x, w);
  const Rows px = c.rows("x", x, x.sizes(), (int64_t)n.H * n.D);
  const float* pw = c.f32("weight", w, w.sizes());
  const void* pdy = c.io("d_y", dy, x.sizes());
  const Out o[3] = {c.out("d_x", a[4], x), c.out("d_weight", a[5], w), c.out("d_bias", a[6], w)};
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[7], api.ttt_backward_layernorm_workspace(c.dt, n.M, n.H, n.D), bytes, held);
  const float eps = number(a[3]);
  const ttt_status st = enqueue(api.ttt_backward_layernorm, c.dt, n.M, n.H, n.D, eps, px.p, px.stride, pw, pdy,
                                o[0].p, (float*)o[1].p, (float*)o[2].p, ws, bytes, c.stream);
  return st == TTT_OK ? tuple_of(o) : status(st);
  END_HANDLE_TH_ERRORS
}

// ---- short causal convolution -----------------------------------------------------------------
struct Conv {
  int B, N, C, K;
};
Conv conv_of(const Tensor& x, const Tensor& weight, bool step) {
  TORCH_CHECK_VALUE(x.dim() == (step ? 2 : 3), step ? "x must be [B, C]" : "x must be [B, N, C]");
  TORCH_CHECK_VALUE(weight.dim() == 2, "weight must be [C, K]");
  const int N = step ? 1 : as_int("x", x.size(1));
  return {as_int("x", x.size(0)), N, as_int("x", x.size(-1)), as_int("weight", weight.size(1))};
}

// (x, weight, bias, silu, state, lengths, state_out, y)
PyObject* conv1d_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(8)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]);
  const Tensor *b = maybe("bias", a[2]), *state = maybe("state", a[4]), *len = maybe("lengths", a[5]);
  const Tensor* so = maybe("state_out", a[6]);
  const Call c("x", x);
  const Conv n = conv_of(x, w, false);
  const int64_t held[3] = {n.B, n.K - 1, n.C};
  const Rows px = c.rows("x", x, x.sizes(), n.C);
  const float *pw = c.f32("weight", w, {n.C, n.K}), *pb = c.f32("bias", b, {n.C});
  const void* ps = c.io("state", state, held);
  const int* pl = c.lengths(len, n.B);
  void* pso = c.io("state_out", so, held);
  const Out y = c.out("y", a[7], x);
  const int silu = truth(a[3]);
  const ttt_status st = enqueue(api.ttt_forward_conv1d, c.dt, n.B, n.N, n.C, n.K, silu, px.p, px.stride, pw, pb, ps,
                                pl, y.p, pso, c.stream);
  if (st == TTT_OK && so) written(*so);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (x, weight, bias, silu, state, state_out, y)
PyObject* conv1d_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(7)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]), &state = tensor_of("state", a[4]);
  const Tensor *b = maybe("bias", a[2]), *so = maybe("state_out", a[5]);
  const Call c("x", x);
  const Conv n = conv_of(x, w, true);
  const int64_t held[3] = {n.B, n.K - 1, n.C};
  const Rows px = c.rows("x", x, x.sizes(), n.C);
  const float *pw = c.f32("weight", w, {n.C, n.K}), *pb = c.f32("bias", b, {n.C});
  void* ps = c.io("state", state, held);
  void* pso = so ? c.io("state_out", *so, held) : ps;
  const Out y = c.out("y", a[6], x);
  const int silu = truth(a[3]);
  const ttt_status st = enqueue(api.ttt_step_conv1d, c.dt, n.B, n.C, n.K, silu, px.p, px.stride, pw, pb, ps, y.p, pso,
                                c.stream);
  if (st == TTT_OK) written(so ? *so : state);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (x, weight, bias, d_y, silu, state, lengths, d_x, d_weight, d_bias, d_state, workspace)
PyObject* conv1d_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(12)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]), &dy = tensor_of("d_y", a[3]);
  const Tensor *b = maybe("bias", a[2]), *state = maybe("state", a[5]), *len = maybe("lengths", a[6]);
  const Call c("x", x);
  const Conv n = conv_of(x, w, false);
  const int64_t held_shape[3] = {n.B, n.K - 1, n.C};
  const Rows px = c.rows("x", x, x.sizes(), n.C);
  const float *pw = c.f32("weight", w, {n.C, n.K}), *pb = c.f32("bias", b, {n.C});
  const void* ps = c.io("state", state, held_shape);
  const int* pl = c.lengths(len, n.B);
  const void* pdy = c.io("d_y", dy, x.sizes());
  const Out o[4] = {c.out("d_x", a[7], x), c.out("d_weight", a[8], w), c.grad("d_bias", a[9], b),
                    c.grad("d_state", a[10], state)};
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[11], api.ttt_backward_conv1d_workspace(c.dt, n.B, n.N, n.C, n.K), bytes, held);
  const int silu = truth(a[4]);
  const ttt_status st = enqueue(api.ttt_backward_conv1d, c.dt, n.B, n.N, n.C, n.K, silu, px.p, px.stride, pw, pb, ps,
                                pl, pdy, o[0].p, (float*)o[1].p, (float*)o[2].p, o[3].p, ws, bytes, c.stream);
  return st == TTT_OK ? tuple_of(o) : status(st);
  END_HANDLE_TH_ERRORS
}

// ---- selective state space scan ---------------------------------------------------------------
// The inputs that every direction starts with: (u, delta, A, Bm, Cm, D, delta_bias, z) at a[0 .. 8).
struct Scan {
  const Tensor &u, &delta, &A, &Bm, &Cm;
  const Tensor *D, *delta_bias, *z;
  int B = 0, N = 1, C = 0, S = 0, G = 0;
  Rows pu, pd, pb, pc, pz;
  const float *pA = nullptr, *pD = nullptr, *pdb = nullptr;

  explicit Scan(PyObject* const* a)
      : u(tensor_of("u", a[0])), delta(tensor_of("delta", a[1])), A(tensor_of("A", a[2])), Bm(tensor_of("Bm", a[3])),
        Cm(tensor_of("Cm", a[4])), D(maybe("D", a[5])), delta_bias(maybe("delta_bias", a[6])), z(maybe("z", a[7])) {}

  void take(const Call& c, bool step) {
    const int lead = step ? 1 : 2;
    TORCH_CHECK_VALUE(u.dim() == lead + 1, step ? "u must be [B, C]" : "u must be [B, N, C]");
    TORCH_CHECK_VALUE(A.dim() == 2, "A must be [C, S]");
    TORCH_CHECK_VALUE(Bm.dim() == lead + 2, step ? "Bm must be [B, G, S]" : "Bm must be [B, N, G, S]");
    B = as_int("u", u.size(0));
    if (!step) N = as_int("u", u.size(1));
    C = as_int("u", u.size(-1)), S = as_int("A", A.size(1)), G = as_int("Bm", Bm.size(-2));
    const int64_t mat4[4] = {B, N, G, S}, mat3[3] = {B, G, S};
    const at::IntArrayRef mat = step ? at::IntArrayRef(mat3, 3) : at::IntArrayRef(mat4, 4);
    pu = c.rows("u", u, u.sizes(), C);
    pd = c.rows("delta", delta, u.sizes(), C);
    pA = c.f32("A", A, {C, S});
    pb = c.rows("Bm", Bm, mat, (int64_t)G * S);
    pc = c.rows("Cm", Cm, mat, (int64_t)G * S);
    pD = c.f32("D", D, {C});
    pdb = c.f32("delta_bias", delta_bias, {C});
    if (z) pz = c.rows("z", *z, u.sizes(), C);
  }
};
#define TTT_SCAN_INPUTS(s)                                                                               \
  s.pu.p, s.pu.stride, s.pd.p, s.pd.stride, s.pA, s.pb.p, s.pb.stride, s.pc.p, s.pc.stride, s.pD, s.pdb, \
      s.pz.p, s.pz.stride

// (inputs, softplus, h0, lengths, h_out, y, workspace)
PyObject* scan_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(14)
  Scan s(a);
  const Tensor *h0 = maybe("h0", a[9]), *len = maybe("lengths", a[10]), *ho = maybe("h_out", a[11]);
  const Call c("u", s.u);
  s.take(c, false);
  const int64_t held_shape[3] = {s.B, s.C, s.S};
  const float *ph = c.f32("h0", h0, held_shape), *pho = c.f32("h_out", ho, held_shape);
  const int* pl = c.lengths(len, s.B);
  const Out y = c.out("y", a[12], s.u);
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[13], api.ttt_forward_selective_scan_workspace(c.dt, s.B, s.N, s.C, s.S, s.G), bytes, held);
  const int softplus = truth(a[8]);
  const ttt_status st = enqueue(api.ttt_forward_selective_scan, c.dt, s.B, s.N, s.C, s.S, s.G, softplus,
                                TTT_SCAN_INPUTS(s), ph, pl, y.p, const_cast<float*>(pho), ws, bytes, c.stream);
  if (st == TTT_OK && ho) written(*ho);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (inputs, softplus, h, h_out, y)
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(12)
  Scan s(a);
  const Tensor& h = tensor_of("h", a[9]);
  const Tensor* ho = maybe("h_out", a[10]);
  const Call c("u", s.u);
  s.take(c, true);
  const int64_t held_shape[3] = {s.B, s.C, s.S};
  const float* ph = c.f32("h", h, held_shape);
  const float* pho = ho ? c.f32("h_out", *ho, held_shape) : ph;
  const Out y = c.out("y", a[11], s.u);
  const int softplus = truth(a[8]);
  const ttt_status st = enqueue(api.ttt_step_selective_scan, c.dt, s.B, s.C, s.S, s.G, softplus, TTT_SCAN_INPUTS(s),
                                ph, y.p, const_cast<float*>(pho), c.stream);
  if (st == TTT_OK) written(ho ? *ho : h);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (inputs, softplus, h0, lengths, d_y, d_u, d_delta, d_A, d_B, d_C, d_D, d_delta_bias, d_z, d_h0, workspace)
PyObject* scan_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(22)
  Scan s(a);
  const Tensor *h0 = maybe("h0", a[9]), *len = maybe("lengths", a[10]);
  const Tensor& dy = tensor_of("d_y", a[11]);
  const Call c("u", s.u);
  s.take(c, false);
  const float* ph = c.f32("h0", h0, {s.B, s.C, s.S});
  const int* pl = c.lengths(len, s.B);
  const void* pdy = c.io("d_y", dy, s.u.sizes());
  const Out o[9] = {c.out("d_u", a[12], s.u),         c.out("d_delta", a[13], s.delta),
                    c.out("d_A", a[14], s.A),         c.out("d_B", a[15], s.Bm),
                    c.out("d_C", a[16], s.Cm),        c.grad("d_D", a[17], s.D),
                    c.grad("d_delta_bias", a[18], s.delta_bias), c.grad("d_z", a[19], s.z),
                    c.grad("d_h0", a[20], h0)};
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[21], api.ttt_backward_selective_scan_workspace(c.dt, s.B, s.N, s.C, s.S, s.G), bytes, held);
  const int softplus = truth(a[8]);
  const ttt_status st = enqueue(api.ttt_backward_selective_scan, c.dt, s.B, s.N, s.C, s.S, s.G, softplus,
                                TTT_SCAN_INPUTS(s), ph, pl, pdy, o[0].p, o[1].p, (float*)o[2].p, o[3].p, o[4].p,
                                (float*)o[5].p, (float*)o[6].p, o[7].p, (float*)o[8].p, ws, bytes, c.stream);
  return st == TTT_OK ? tuple_of(o) : status(st);
  END_HANDLE_TH_ERRORS
}

// bind(handle): looks the entry points up in a loaded libttt.so.
PyObject* bind(PyObject*, PyObject* handle) {
  void* lib = PyLong_AsVoidPtr(handle);
  if (PyErr_Occurred()) return nullptr;
#define TTT_FN(name)                                                              \
  if (!(api.name = reinterpret_cast<decltype(api.name)>(dlsym(lib, #name)))) {    \
    PyErr_SetString(PyExc_RuntimeError, "libttt.so lacks " #name);                \
    return nullptr;                                                               \
  }
  TTT_FN(ttt_forward_layernorm)
  TTT_FN(ttt_backward_layernorm)
  TTT_FN(ttt_backward_layernorm_workspace)
  TTT_FN(ttt_forward_conv1d)
  TTT_FN(ttt_step_conv1d)
  TTT_FN(ttt_backward_conv1d)
  TTT_FN(ttt_backward_conv1d_workspace)
  TTT_FN(ttt_forward_selective_scan)
  TTT_FN(ttt_forward_selective_scan_workspace)
  TTT_FN(ttt_step_selective_scan)
  TTT_FN(ttt_backward_selective_scan)
  TTT_FN(ttt_backward_selective_scan_workspace)
#undef TTT_FN
  Py_RETURN_NONE;
}

#define TTT_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         TTT_METHOD(layernorm_forward),
                         TTT_METHOD(layernorm_backward),
                         TTT_METHOD(conv1d_forward),
                         TTT_METHOD(conv1d_step),
                         TTT_METHOD(conv1d_backward),
                         TTT_METHOD(scan_forward),
                         TTT_METHOD(scan_step),
                         TTT_METHOD(scan_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_seq_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seq_native() { return PyModule_Create(&module); }
