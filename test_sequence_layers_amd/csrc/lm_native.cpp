// The marshalling of lm.py, the second part of the extension module _seq_native (seq_native.cpp): tensors in, the C
// ABI of include/ttt_lm.h called on the current stream, tensors out.
#include "../../include/ttt_lm.h"
#include "native.hpp"

namespace {

struct Api {
#define TTT_FN(name) decltype(&::name) name
  TTT_FN(ttt_forward_rmsnorm);
  TTT_FN(ttt_forward_rmsnorm_e4m3);
  TTT_FN(ttt_backward_rmsnorm);
  TTT_FN(ttt_backward_rmsnorm_workspace);
  TTT_FN(ttt_forward_dropout);
  TTT_FN(ttt_backward_dropout);
  TTT_FN(ttt_forward_gated_recurrence);
  TTT_FN(ttt_forward_gated_recurrence_workspace);
  TTT_FN(ttt_step_gated_recurrence);
  TTT_FN(ttt_backward_gated_recurrence);
  TTT_FN(ttt_backward_gated_recurrence_workspace);
#undef TTT_FN
} api;

// p and, where it drops, rng: int64 [2].
struct Dropping {
  double p;
  const long long* rng = nullptr;
  Dropping(const Call& c, PyObject* p_, PyObject* rng_) : p(real(p_)) {
    if (p == 0.0) return;
    TORCH_CHECK_VALUE(rng_ != Py_None, "dropout (p other than 0) needs rng");
    rng = static_cast<const long long*>(c.need("rng", tensor_of("rng", rng_), {2}, at::kLong));
  }
};

// ---- RMS norm ---------------------------------------------------------------------------------
// (x, weight, eps, residual, p, rng, sum_out, y)
PyObject* rmsnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(8)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]);
  const Tensor* res = maybe("residual", a[3]);
  const Call c("x", x);
  const Norm n = norm_of(x, w);
  const Rows px = c.rows("x", x, x.sizes(), (int64_t)n.H * n.D);
  const float* pw = c.f32("weight", w, w.sizes());
  const void* pr = c.io("residual", res, x.sizes());
  const Dropping d(c, a[4], a[5]);
  const Out o[2] = {c.out("y", a[7], x), c.grad("sum_out", a[6], res)};
  const float eps = number(a[2]);
  const ttt_status st = enqueue(api.ttt_forward_rmsnorm, c.dt, n.M, n.H, n.D, eps, px.p, px.stride, pr, d.p, d.rng, pw,
                                o[1].p, o[0].p, c.stream);
  if (st != TTT_OK) return status(st);
  return res ? tuple_of(o) : o[0].object();
  END_HANDLE_TH_ERRORS
}

// (x, weight, eps, residual, group, sum_out, y, scales)
PyObject* rmsnorm_e4m3(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(8)
  const Tensor &x = tensor_of("x", a[0]), &w = tensor_of("weight", a[1]);
  const Tensor* res = maybe("residual", a[3]);
  const Call c("x", x);
  const Norm n = norm_of(x, w);
  const Rows px = c.rows("x", x, x.sizes(), (int64_t)n.H * n.D);
  const float* pw = c.f32("weight", w, w.sizes());
  const void* pr = c.io("residual", res, x.sizes());
  const long asked = PyLong_AsLong(a[4]);
  if (asked == -1 && PyErr_Occurred()) throw python_error();
  const int group = asked == 0 ? n.D : as_int("group", asked);
  TORCH_CHECK_VALUE(group > 0 && n.D % group == 0, "group must divide ", n.D);
  auto shape = x.sizes().vec();
  shape.back() = n.D / group;
  const Out y = c.out("y", a[6], x.sizes(), at::kFloat8_e4m3fn), scales = c.out("scales", a[7], shape, at::kFloat);
  const Out sum = c.grad("sum_out", a[5], res);
  const float eps = number(a[2]);
  const ttt_status st = enqueue(api.ttt_forward_rmsnorm_e4m3, c.dt, n.M, n.H, n.D, group, eps, px.p, px.stride, pr, pw,
                                sum.p, y.p, (float*)scales.p, c.stream);
  if (st != TTT_OK) return status(st);
  return res ? tuple_of({y, scales, sum}) : tuple_of({y, scales});
  END_HANDLE_TH_ERRORS
}

// (s, weight, d_y, eps, d_sum, p, rng, d_s, d_x, d_weight, workspace)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(11)
  const Tensor &s = tensor_of("s", a[0]), &w = tensor_of("weight", a[1]), &dy = tensor_of("d_y", a[2]);
  const Tensor* dsum = maybe("d_sum", a[4]);
  const Call c("s", s);
  const Norm n = norm_of(s, w);
  const Rows ps = c.rows("s", s, s.sizes(), (int64_t)n.H * n.D);
  const float* pw = c.f32("weight", w, w.sizes());
  const void *pdy = c.io("d_y", dy, s.sizes()), *pds = c.io("d_sum", dsum, s.sizes());
  const Dropping d(c, a[5], a[6]);
  const Out o[3] = {c.out("d_s", a[7], s), c.grad("d_x", a[8], d.p != 0.0 ? &s : nullptr), c.out("d_weight", a[9], w)};
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[10], api.ttt_backward_rmsnorm_workspace(c.dt, n.M, n.H, n.D), bytes, held);
  const float eps = number(a[3]);
  const ttt_status st = enqueue(api.ttt_backward_rmsnorm, c.dt, n.M, n.H, n.D, eps, ps.p, ps.stride, pw, pdy, pds, d.p,
                                d.rng, o[0].p, o[1].p, (float*)o[2].p, ws, bytes, c.stream);
  return st == TTT_OK ? tuple_of(o) : status(st);
  END_HANDLE_TH_ERRORS
}

// ---- dropout ----------------------------------------------------------------------------------
// Rows of the last dim.
struct Matrix {
  int M, C;
};
Matrix matrix_of(const char* name, const Tensor& x) {
  TORCH_CHECK_VALUE(x.dim() >= 1, name, " must have a dim");
  const int64_t C = x.size(-1);
  return {as_int(name, C ? x.numel() / C : 0), as_int(name, C)};
}

// (x, p, rng, residual, y)
PyObject* dropout_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(5)
  const Tensor& x = tensor_of("x", a[0]);
  const Tensor* res = maybe("residual", a[3]);
  const Call c("x", x);
  const Matrix m = matrix_of("x", x);
  const Rows px = c.rows("x", x, x.sizes(), m.C);
  const void* pr = c.io("residual", res, x.sizes());
  const Dropping d(c, a[1], a[2]);
  const Out y = c.out("y", a[4], x);
  const ttt_status st = enqueue(api.ttt_forward_dropout, c.dt, m.M, m.C, d.p, d.rng, px.p, px.stride, pr, y.p, c.stream);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (d_y, p, rng, d_x)
PyObject* dropout_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(4)
  const Tensor& dy = tensor_of("d_y", a[0]);
  const Call c("d_y", dy);
  const Matrix m = matrix_of("d_y", dy);
  const void* pdy = c.io("d_y", dy, dy.sizes());
  const Dropping d(c, a[1], a[2]);
  const Out dx = c.out("d_x", a[3], dy);
  const ttt_status st = enqueue(api.ttt_backward_dropout, c.dt, m.M, m.C, d.p, d.rng, pdy, dx.p, c.stream);
  return st == TTT_OK ? dx.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// ---- gated recurrence -------------------------------------------------------------------------
// The inputs that every direction starts with: (x, r, i, lam) at a[0 .. 4).
struct Gated {
  const Tensor &x, &r, &i, &lam;
  int B = 0, N = 1, C = 0;
  Rows px, pr, pi;
  const float* pl = nullptr;

  explicit Gated(PyObject* const* a)
      : x(tensor_of("x", a[0])), r(tensor_of("r", a[1])), i(tensor_of("i", a[2])), lam(tensor_of("lam", a[3])) {}

  void take(const Call& c, bool step) {
    TORCH_CHECK_VALUE(x.dim() == (step ? 2 : 3), step ? "x must be [B, C]" : "x must be [B, N, C]");
    B = as_int("x", x.size(0));
    if (!step) N = as_int("x", x.size(1));
    C = as_int("x", x.size(-1));
    px = c.rows("x", x, x.sizes(), C);
    pr = c.rows("r", r, x.sizes(), C);
    pi = c.rows("i", i, x.sizes(), C);
    pl = c.f32("lam", lam, {C});
  }
};
#define TTT_GATED_INPUTS(g) g.px.p, g.px.stride, g.pr.p, g.pr.stride, g.pi.p, g.pi.stride, g.pl

// (inputs, scale, h0, lengths, states, h_out, y, workspace)
PyObject* recurrence_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(11)
  Gated g(a);
  const Tensor *h0 = maybe("h0", a[5]), *len = maybe("lengths", a[6]), *kept = maybe("states", a[7]);
  const Tensor* ho = maybe("h_out", a[8]);
  const Call c("x", g.x);
  g.take(c, false);
  const int64_t held_shape[2] = {g.B, g.C}, kept_shape[3] = {g.B, ((int64_t)g.N + 63) / 64, g.C};
  const float *ph = c.f32("h0", h0, held_shape), *pho = c.f32("h_out", ho, held_shape);
  const float* pk = c.f32("states", kept, kept_shape);
  const int* pl = c.lengths(len, g.B);
  const Out y = c.out("y", a[9], g.x);
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[10], api.ttt_forward_gated_recurrence_workspace(c.dt, g.B, g.N, g.C), bytes, held);
  const float scale = number(a[4]);
  const ttt_status st = enqueue(api.ttt_forward_gated_recurrence, c.dt, g.B, g.N, g.C, scale, TTT_GATED_INPUTS(g), ph, pl,
                                y.p, const_cast<float*>(pk), const_cast<float*>(pho), ws, bytes, c.stream);
  if (st == TTT_OK && kept) written(*kept);
  if (st == TTT_OK && ho) written(*ho);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (inputs, scale, h, h_out, y)
PyObject* recurrence_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(8)
  Gated g(a);
  const Tensor& h = tensor_of("h", a[5]);
  const Tensor* ho = maybe("h_out", a[6]);
  const Call c("x", g.x);
  g.take(c, true);
  const int64_t held_shape[2] = {g.B, g.C};
  const float* ph = c.f32("h", h, held_shape);
  const float* pho = ho ? c.f32("h_out", *ho, held_shape) : ph;
  const Out y = c.out("y", a[7], g.x);
  const float scale = number(a[4]);
  const ttt_status st = enqueue(api.ttt_step_gated_recurrence, c.dt, g.B, g.C, scale, TTT_GATED_INPUTS(g), ph, y.p,
                                const_cast<float*>(pho), c.stream);
  if (st == TTT_OK) written(ho ? *ho : h);
  return st == TTT_OK ? y.object() : status(st);
  END_HANDLE_TH_ERRORS
}

// (inputs, scale, h0, lengths, states, d_y, d_x, d_r, d_i, d_lam, d_h0, workspace)
PyObject* recurrence_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  TTT_ARGS(15)
  Gated g(a);
  const Tensor *h0 = maybe("h0", a[5]), *len = maybe("lengths", a[6]), *kept = maybe("states", a[7]);
  const Tensor& dy = tensor_of("d_y", a[8]);
  const Call c("x", g.x);
  g.take(c, false);
  const int64_t held_shape[2] = {g.B, g.C}, kept_shape[3] = {g.B, ((int64_t)g.N + 63) / 64, g.C};
  const float *ph = c.f32("h0", h0, held_shape), *pk = c.f32("states", kept, kept_shape);
  const int* pl = c.lengths(len, g.B);
  const void* pdy = c.io("d_y", dy, g.x.sizes());
  const Out o[5] = {c.out("d_x", a[9], g.x), c.out("d_r", a[10], g.r), c.out("d_i", a[11], g.i),
                    c.out("d_lam", a[12], g.lam), c.grad("d_h0", a[13], h0)};
  size_t bytes;
  c10::DataPtr held;
  void* ws = c.workspace(a[14], api.ttt_backward_gated_recurrence_workspace(c.dt, g.B, g.N, g.C, pk != nullptr), bytes, held);
  const float scale = number(a[4]);
  const ttt_status st = enqueue(api.ttt_backward_gated_recurrence, c.dt, g.B, g.N, g.C, scale, TTT_GATED_INPUTS(g), ph, pl,
                                pk, pdy, o[0].p, o[1].p, o[2].p, (float*)o[3].p, (float*)o[4].p, ws, bytes, c.stream);
  return st == TTT_OK ? tuple_of(o) : status(st);
  END_HANDLE_TH_ERRORS
}

}  // namespace

bool lm_bind(void* lib) {
  const bool failed = false;
  TTT_LOOKUP(ttt_forward_rmsnorm)
  TTT_LOOKUP(ttt_forward_rmsnorm_e4m3)
  TTT_LOOKUP(ttt_backward_rmsnorm)
  TTT_LOOKUP(ttt_backward_rmsnorm_workspace)
  TTT_LOOKUP(ttt_forward_dropout)
  TTT_LOOKUP(ttt_backward_dropout)
  TTT_LOOKUP(ttt_forward_gated_recurrence)
  TTT_LOOKUP(ttt_forward_gated_recurrence_workspace)
  TTT_LOOKUP(ttt_step_gated_recurrence)
  TTT_LOOKUP(ttt_backward_gated_recurrence)
  TTT_LOOKUP(ttt_backward_gated_recurrence_workspace)
  return true;
}

PyMethodDef lm_methods[] = {TTT_METHOD(rmsnorm_forward),    TTT_METHOD(rmsnorm_e4m3),       TTT_METHOD(rmsnorm_backward),
                            TTT_METHOD(dropout_forward),    TTT_METHOD(dropout_backward),   TTT_METHOD(recurrence_forward),
                            TTT_METHOD(recurrence_step),    TTT_METHOD(recurrence_backward), {nullptr, nullptr, 0, nullptr}};
