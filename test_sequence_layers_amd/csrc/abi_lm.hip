// C ABI of the residual block's operators (include/ttt_lm.h): argument validation, workspace sizing and dispatch.
// Every check runs before anything is enqueued, so a failed call leaves the outputs untouched.
#include <math.h>
#include <stdint.h>

#include "../../include/ttt_lm.h"
#include "abi_checks.hpp"
#include "internal.hpp"
#include "lm.hpp"

namespace {

using ttt::kKept;
using ttt::round_up;

ttt_status check_rmsnorm_sizes(ttt_dtype dt, int M, int H, int D) {
  if (!known(dt) || M <= 0 || H <= 0 || D <= 0) return TTT_ERR_INVALID;
  if (D > 16384 || H > 65535 || (long long)H * D > (1 << 24) || (long long)M * H > 0x7fffffffll)
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

ttt_status check_recurrence_sizes(ttt_dtype dt, int B, int N, int C) {
  if (!known(dt) || B <= 0 || N <= 0 || C <= 0) return TTT_ERR_INVALID;
  if (B > kMaxB || N > (1 << 22) || C > (1 << 20) || (double)B * (N + 128.) * (C + 64.) > (double)(1ll << 38))
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// What p and rng say; false where they are refused.
bool drop_of(double p, const long long* rng, ttt::Drop* d) {
  if (!(p >= 0. && p < 1.)) return false;
  const double least = rint(p * 65536.);
  if (least >= 65536.) return false;
  *d = ttt::Drop{reinterpret_cast<const unsigned long long*>(rng), (uint32_t)least, (float)(65536. / (65536. - least))};
  return true;
}

void add_rng(Buffers& bufs, double p, const long long* rng) {
  if (p > 0.) bufs.in(rng, 16, 8);
}

bool positive(float v) { return isfinite(v) && v > 0.f; }

ttt_status forward_rmsnorm(ttt_dtype dt, double p, const long long* rng, ttt::RmsNormArgs& a, bool e4m3, void* stream) {
  const ttt_status st = check_rmsnorm_sizes(dt, a.M, a.H, a.D);
  if (st != TTT_OK) return st;
  if (!isfinite(a.eps) || a.eps < 0.f || !drop_of(p, rng, &a.drop) || !a.residual != !a.sum || (p > 0. && !a.residual))
    return TTT_ERR_INVALID;
  const bool parts = a.group != a.D;
  if (a.group <= 0 || a.D % a.group != 0) return TTT_ERR_INVALID;
  if ((parts && a.group != 32 && a.group != 64 && a.group != 128) || (a.residual && a.H != 1)) return TTT_ERR_UNSUPPORTED;
  const size_t e = elem_size(dt), n = (size_t)a.M * a.H * a.D;
  Buffers bufs;
  bufs.rows(a.x, a.M, a.xs, (long long)a.H * a.D, e);
  bufs.in(a.w, (size_t)a.H * a.D * 4, 4);
  if (a.residual != a.sum) bufs.in(a.residual, n * e, e);
  bufs.out(a.sum, n * e, e, false);
  bufs.out(a.y, e4m3 ? n : n * e, e4m3 ? 1 : e);
  if (e4m3) bufs.out(a.scales, n / a.group * 4, 4);
  add_rng(bufs, p, rng);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::rmsnorm_launch(dt == TTT_BF16, a, static_cast<hipStream_t>(stream)));
}

// The inputs every direction of the recurrence reads.
void add_recurrence_inputs(Buffers& bufs, ttt_dtype dt, const ttt::RecurrenceArgs& a) {
  const size_t e = elem_size(dt);
  const long long t = (long long)a.B * a.N;
  bufs.rows(a.x, t, a.xs, a.C, e);
  bufs.rows(a.r, t, a.rs, a.C, e);
  bufs.rows(a.i, t, a.is, a.C, e);
  bufs.in(a.lam, (size_t)a.C * 4, 4);
  bufs.in(a.lengths, (size_t)a.B * 4, 4, false);
}
size_t kept_bytes(int B, int N, int C) { return (size_t)B * ((N + kKept - 1) / kKept) * C * 4; }

}  // namespace

extern "C" {

ttt_status ttt_forward_rmsnorm(ttt_dtype dt, int M, int H, int D, float eps, const void* x, long long x_stride,
                               const void* residual, double p, const long long* rng, const float* weight, void* sum,
                               void* y, void* stream) {
  ttt::RmsNormArgs a{};
  a.M = M, a.H = H, a.D = D, a.group = D, a.eps = eps, a.x = x, a.xs = x_stride, a.w = weight, a.residual = residual;
  a.sum = sum, a.y = y;
  return forward_rmsnorm(dt, p, rng, a, false, stream);
}

ttt_status ttt_forward_rmsnorm_e4m3(ttt_dtype dt, int M, int H, int D, int group, float eps, const void* x,
                                    long long x_stride, const void* residual, const float* weight, void* sum, void* y,
                                    float* scales, void* stream) {
  ttt::RmsNormArgs a{};
  a.M = M, a.H = H, a.D = D, a.group = group, a.eps = eps, a.x = x, a.xs = x_stride, a.w = weight, a.residual = residual;
  a.sum = sum, a.y = y, a.scales = scales;
  return forward_rmsnorm(dt, 0., nullptr, a, true, stream);
}

size_t ttt_backward_rmsnorm_workspace(ttt_dtype dt, int M, int H, int D) {
  if (check_rmsnorm_sizes(dt, M, H, D) != TTT_OK) return 0;
  return round_up(ttt::rmsnorm_bwd_workspace_bytes(dt == TTT_BF16, M, H, D), 256);
}

ttt_status ttt_backward_rmsnorm(ttt_dtype dt, int M, int H, int D, float eps, const void* s, long long s_stride,
                                const float* weight, const void* d_y, const void* d_sum, double p, const long long* rng,
                                void* d_s, void* d_x, float* d_weight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  ttt_status st = check_rmsnorm_sizes(dt, M, H, D);
  if (st != TTT_OK) return st;
  ttt::RmsNormArgs a{};
  if (!isfinite(eps) || eps < 0.f || !drop_of(p, rng, &a.drop) || (p > 0.) != (d_x != nullptr)) return TTT_ERR_INVALID;
  if (p > 0. && H != 1) return TTT_ERR_UNSUPPORTED;
  a.M = M, a.H = H, a.D = D, a.eps = eps, a.x = s, a.xs = s_stride, a.w = weight, a.dy = d_y, a.dsum = d_sum, a.ds = d_s;
  a.dx = d_x, a.dw = d_weight, a.partial = static_cast<float*>(workspace);
  const size_t e = elem_size(dt), par = (size_t)H * D * sizeof(float), act = (size_t)M * H * D * e;
  Buffers bufs;
  bufs.rows(s, M, s_stride, (long long)H * D, e);
  bufs.in(weight, par, 4);
  bufs.in(d_y, act, e);
  if (d_sum != d_s) bufs.in(d_sum, act, e, false);
  bufs.out(d_s, act, e);
  bufs.out(d_x, act, e, false);
  bufs.out(d_weight, par, 4);
  add_rng(bufs, p, rng);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_backward_rmsnorm_workspace(dt, M, H, D));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::rmsnorm_bwd_launch(dt == TTT_BF16, a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_forward_dropout(ttt_dtype dt, int M, int C, double p, const long long* rng, const void* x,
                               long long x_stride, const void* residual, void* y, void* stream) {
  if (!known(dt) || M <= 0 || C <= 0) return TTT_ERR_INVALID;
  if (C > (1 << 24) || (double)M * C > (double)(1ll << 46)) return TTT_ERR_UNSUPPORTED;
  ttt::DropoutArgs a{};
  a.M = M, a.C = C, a.x = x, a.xs = x_stride, a.residual = residual, a.y = y;
  if (!drop_of(p, rng, &a.drop)) return TTT_ERR_INVALID;
  const size_t e = elem_size(dt), n = (size_t)M * C * e;
  Buffers bufs;
  if (x != y || x_stride != C) bufs.rows(x, M, x_stride, C, e);
  if (residual != y) bufs.in(residual, n, e, false);
  bufs.out(y, n, e);
  add_rng(bufs, p, rng);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::dropout_launch(dt == TTT_BF16, a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_backward_dropout(ttt_dtype dt, int M, int C, double p, const long long* rng, const void* d_y, void* d_x,
                                void* stream) {
  return ttt_forward_dropout(dt, M, C, p, rng, d_y, C, nullptr, d_x, stream);
}

long long ttt_dropout_counters(int M, int C) { return M <= 0 || C <= 0 ? 0 : (long long)M * (((long long)C + 7) / 8); }

size_t ttt_forward_gated_recurrence_workspace(ttt_dtype dt, int B, int N, int C) {
  if (check_recurrence_sizes(dt, B, N, C) != TTT_OK) return 0;
  return round_up(ttt::recurrence_workspace_bytes(dt == TTT_BF16, B, N, C), 256);
}

ttt_status ttt_forward_gated_recurrence(ttt_dtype dt, int B, int N, int C, float scale, const void* x,
                                        long long x_stride, const void* r, long long r_stride, const void* i,
                                        long long i_stride, const float* lam, const float* h0, const int* lengths,
                                        void* y, float* states, float* h_out, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  ttt_status st = check_recurrence_sizes(dt, B, N, C);
  if (st != TTT_OK) return st;
  if (!positive(scale)) return TTT_ERR_INVALID;
  ttt::RecurrenceArgs a{};
  a.B = B, a.N = N, a.C = C, a.scale = scale, a.x = x, a.r = r, a.i = i, a.xs = x_stride, a.rs = r_stride, a.is = i_stride;
  a.lam = lam, a.h0 = h0, a.lengths = lengths, a.y = y, a.states = states, a.h_out = h_out;
  const size_t e = elem_size(dt), held = (size_t)B * C * 4;
  Buffers bufs;
  add_recurrence_inputs(bufs, dt, a);
  bufs.in(h0, held, 4, false);
  bufs.out(y, (size_t)B * N * C * e, e);
  bufs.out(states, kept_bytes(B, N, C), 4, false);
  bufs.out(h_out, held, 4, false);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_forward_gated_recurrence_workspace(dt, B, N, C));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::recurrence_launch(dt == TTT_BF16, a, workspace, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_step_gated_recurrence(ttt_dtype dt, int B, int C, float scale, const void* x, long long x_stride,
                                     const void* r, long long r_stride, const void* i, long long i_stride,
                                     const float* lam, const float* h, void* y, float* h_out, void* stream) {
  const ttt_status st = check_recurrence_sizes(dt, B, 1, C);
  if (st != TTT_OK) return st;
  if (!positive(scale)) return TTT_ERR_INVALID;
  ttt::RecurrenceArgs a{};
  a.B = B, a.N = 1, a.C = C, a.scale = scale, a.x = x, a.r = r, a.i = i, a.xs = x_stride, a.rs = r_stride, a.is = i_stride;
  a.lam = lam, a.h0 = h, a.y = y, a.h_out = h_out;
  const size_t e = elem_size(dt), held = (size_t)B * C * 4;
  Buffers bufs;
  add_recurrence_inputs(bufs, dt, a);
  if (h != h_out) bufs.in(h, held, 4);
  bufs.out(h_out, held, 4);
  bufs.out(y, (size_t)B * C * e, e);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::recurrence_step_launch(dt == TTT_BF16, a, static_cast<hipStream_t>(stream)));
}

size_t ttt_backward_gated_recurrence_workspace(ttt_dtype dt, int B, int N, int C, int states) {
  if (check_recurrence_sizes(dt, B, N, C) != TTT_OK) return 0;
  return round_up(ttt::recurrence_bwd_workspace_bytes(dt == TTT_BF16, B, N, C, states != 0), 256);
}

ttt_status ttt_backward_gated_recurrence(ttt_dtype dt, int B, int N, int C, float scale, const void* x,
                                         long long x_stride, const void* r, long long r_stride, const void* i,
                                         long long i_stride, const float* lam, const float* h0, const int* lengths,
                                         const float* states, const void* d_y, void* d_x, void* d_r, void* d_i,
                                         float* d_lam, float* d_h0, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  ttt_status st = check_recurrence_sizes(dt, B, N, C);
  if (st != TTT_OK) return st;
  if (!positive(scale)) return TTT_ERR_INVALID;
  ttt::RecurrenceArgs a{};
  a.B = B, a.N = N, a.C = C, a.scale = scale, a.x = x, a.r = r, a.i = i, a.xs = x_stride, a.rs = r_stride, a.is = i_stride;
  a.lam = lam, a.h0 = h0, a.lengths = lengths, a.kept = states, a.dy = d_y, a.dx = d_x, a.dr = d_r, a.di = d_i;
  a.dlam = d_lam, a.dh0 = d_h0;
  const size_t e = elem_size(dt), held = (size_t)B * C * 4, act = (size_t)B * N * C * e;
  Buffers bufs;
  add_recurrence_inputs(bufs, dt, a);
  bufs.in(h0, held, 4, false);
  bufs.in(states, kept_bytes(B, N, C), 4, false);
  bufs.in(d_y, act, e);
  bufs.out(d_x, act, e);
  bufs.out(d_r, act, e);
  bufs.out(d_i, act, e);
  bufs.out(d_lam, (size_t)C * 4, 4);
  bufs.out(d_h0, held, 4, false);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_backward_gated_recurrence_workspace(dt, B, N, C, states != nullptr));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::recurrence_bwd_launch(dt == TTT_BF16, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
