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
#include "../../include/ttt_seq.h"
#include "native.hpp"

namespace {

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

// ---- layer norm -------------------------------------------------------------------------------
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
  PyObject* const failed = nullptr;
  TTT_LOOKUP(ttt_forward_layernorm)
  TTT_LOOKUP(ttt_backward_layernorm)
  TTT_LOOKUP(ttt_backward_layernorm_workspace)
  TTT_LOOKUP(ttt_forward_conv1d)
  TTT_LOOKUP(ttt_step_conv1d)
  TTT_LOOKUP(ttt_backward_conv1d)
  TTT_LOOKUP(ttt_backward_conv1d_workspace)
  TTT_LOOKUP(ttt_forward_selective_scan)
  TTT_LOOKUP(ttt_forward_selective_scan_workspace)
  TTT_LOOKUP(ttt_step_selective_scan)
  TTT_LOOKUP(ttt_backward_selective_scan)
  TTT_LOOKUP(ttt_backward_selective_scan_workspace)
  if (!lm_bind(lib)) return nullptr;
  Py_RETURN_NONE;
}

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

PyMODINIT_FUNC PyInit__seq_native() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddFunctions(m, lm_methods) < 0) Py_CLEAR(m);
  return m;
}
