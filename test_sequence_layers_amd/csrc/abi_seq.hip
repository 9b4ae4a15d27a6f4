// C ABI of the block operators (include/ttt_seq.h): argument validation, workspace sizing and dispatch.
// Every check runs before anything is enqueued, so a failed call leaves the outputs untouched.
#include <math.h>
#include <stdint.h>

#include "../../include/ttt_seq.h"
#include "internal.hpp"
#include "seq.hpp"

namespace {

using ttt::round_up;

constexpr int kMaxB = 65535;

bool known(ttt_dtype dt) { return dt == TTT_F32 || dt == TTT_BF16; }
size_t elem_size(ttt_dtype dt) { return dt == TTT_BF16 ? 2 : 4; }
ttt_status from_hip(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_HIP; }

// The buffers of one call: alignment and presence are noted as they are added, overlaps (of any
// output with anything but itself) are looked for at the end.
class Buffers {
 public:
  void in(const void* p, size_t bytes, size_t align, bool needed = true) { add(p, bytes, align, needed, false); }
  void out(const void* p, size_t bytes, size_t align, bool needed = true) { add(p, bytes, align, needed, true); }
  // rows tokens of `width` elements, `stride` apart.
  void rows(const void* p, long long rows, long long stride, long long width, size_t e, bool needed = true) {
    if (p && (stride < width || (double)rows * (double)stride > (double)(1ll << 46))) bad_ = true;
    else in(p, ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * e, e, needed);
  }
  bool ok() const {
    if (bad_) return false;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((b_[i].out || b_[j].out) && b_[i].lo < b_[j].hi && b_[j].lo < b_[i].hi) return false;
    return true;
  }

 private:
  void add(const void* p, size_t bytes, size_t align, bool needed, bool out) {
    if (!p) {
      bad_ = bad_ || needed;
      return;
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a & (align - 1)) bad_ = true;
    b_[n_++] = Buf{a, a + bytes, out};
  }
  struct Buf {
    uintptr_t lo, hi;
    bool out;
  };
  Buf b_[24];
  int n_ = 0;
  bool bad_ = false;
};

// Workspace: TTT_ERR_WORKSPACE when it is missing or small, otherwise added as an output (16-byte
// aligned) so that it overlaps nothing.
ttt_status add_workspace(Buffers& bufs, void* ws, size_t have, size_t need) {
  if (need == 0) return TTT_OK;
  if (!ws || have < need) return TTT_ERR_WORKSPACE;
  bufs.out(ws, need, 16);
  return TTT_OK;
}

ttt_status check_layernorm_sizes(ttt_dtype dt, int M, int H, int D) {
  if (!known(dt) || M <= 0 || H <= 0 || D <= 0) return TTT_ERR_INVALID;
  if (D > 16384 || H > 65535 || (long long)H * D > (1 << 24) || (long long)M * H > 0x7fffffffll)
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

ttt_status check_conv1d_sizes(ttt_dtype dt, int B, int N, int C, int K) {
  if (!known(dt) || B <= 0 || N <= 0 || C <= 0 || K <= 0) return TTT_ERR_INVALID;
  if (K < 2 || K > 4 || B > kMaxB || N > (1 << 22) || C > (1 << 20)) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

ttt_status check_scan_sizes(ttt_dtype dt, int B, int N, int C, int S, int G) {
  if (!known(dt) || B <= 0 || N <= 0 || C <= 0 || S <= 0 || G <= 0 || C % G != 0) return TTT_ERR_INVALID;
  if (!ttt::scan_supported_s(S) || B > kMaxB || N > (1 << 22) || C > (1 << 20) ||
      (double)B * C * ((double)N + 4096.) > (double)(1ll << 38) ||
      (long long)B * G * ((C / G + 63) / 64) > (1 << 20))
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// The inputs every direction of the scan reads.
void add_scan_inputs(Buffers& bufs, ttt_dtype dt, int B, int N, int S, const ttt::ScanArgs& a) {
  const size_t e = elem_size(dt);
  const long long t = (long long)B * N;
  bufs.rows(a.u, t, a.us, a.C, e);
  bufs.rows(a.delta, t, a.ds, a.C, e);
  bufs.rows(a.z, t, a.zs, a.C, e, false);
  bufs.rows(a.bm, t, a.bs, (long long)a.G * S, e);
  bufs.rows(a.cm, t, a.cs, (long long)a.G * S, e);
  bufs.in(a.A, (size_t)a.C * S * 4, 4);
  bufs.in(a.D, (size_t)a.C * 4, 4, false);
  bufs.in(a.dbias, (size_t)a.C * 4, 4, false);
  bufs.in(a.lengths, (size_t)B * 4, 4, false);
}

// Bm and Cm are read by scalar loads of whole dwords.
bool dword_rows(const ttt::ScanArgs& a, ttt_dtype dt) {
  if (dt != TTT_BF16) return true;
  return ((reinterpret_cast<uintptr_t>(a.bm) | reinterpret_cast<uintptr_t>(a.cm)) & 3u) == 0 &&
         ((a.bs | a.cs) & 1) == 0;
}

}  // namespace

extern "C" {

ttt_status ttt_forward_layernorm(ttt_dtype dt, int M, int H, int D, float eps, const void* x,
                                 long long x_stride, const float* weight, const float* bias,
                                 void* y, void* stream) {
  const ttt_status st = check_layernorm_sizes(dt, M, H, D);
  if (st != TTT_OK) return st;
  if (!isfinite(eps) || eps < 0.f) return TTT_ERR_INVALID;
  const size_t e = elem_size(dt), par = (size_t)H * D * sizeof(float);
  Buffers bufs;
  bufs.rows(x, M, x_stride, (long long)H * D, e);
  bufs.in(weight, par, 4);
  bufs.in(bias, par, 4, false);
  bufs.out(y, (size_t)M * H * D * e, e);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::layernorm_launch(dt == TTT_BF16, M, H, D, eps, x, x_stride, weight, bias, y,
                                        static_cast<hipStream_t>(stream)));
}

size_t ttt_backward_layernorm_workspace(ttt_dtype dt, int M, int H, int D) {
  if (check_layernorm_sizes(dt, M, H, D) != TTT_OK) return 0;
  return round_up(ttt::layernorm_bwd_workspace_bytes(dt == TTT_BF16, M, H, D), 256);
}

ttt_status ttt_backward_layernorm(ttt_dtype dt, int M, int H, int D, float eps, const void* x,
                                  long long x_stride, const float* weight, const void* d_y,
                                  void* d_x, float* d_weight, float* d_bias, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  ttt_status st = check_layernorm_sizes(dt, M, H, D);
  if (st != TTT_OK) return st;
  if (!isfinite(eps) || eps < 0.f) return TTT_ERR_INVALID;
  const size_t e = elem_size(dt), par = (size_t)H * D * sizeof(float), act = (size_t)M * H * D * e;
  Buffers bufs;
  bufs.rows(x, M, x_stride, (long long)H * D, e);
  bufs.in(weight, par, 4);
  bufs.in(d_y, act, e);
  bufs.out(d_x, act, e);
  bufs.out(d_weight, par, 4);
  bufs.out(d_bias, par, 4, false);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_backward_layernorm_workspace(dt, M, H, D));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::layernorm_bwd_launch(dt == TTT_BF16, M, H, D, eps, x, x_stride, weight, d_y, d_x,
                                            d_weight, d_bias, workspace, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_forward_conv1d(ttt_dtype dt, int B, int N, int C, int K, int silu, const void* x,
                              long long x_stride, const float* weight, const float* bias,
                              const void* state, const int* lengths, void* y, void* state_out,
                              void* stream) {
  const ttt_status st = check_conv1d_sizes(dt, B, N, C, K);
  if (st != TTT_OK) return st;
  if (silu != 0 && silu != 1) return TTT_ERR_INVALID;
  const size_t e = elem_size(dt), held = (size_t)B * (K - 1) * C * e;
  Buffers bufs;
  bufs.rows(x, (long long)B * N, x_stride, C, e);
  bufs.in(weight, (size_t)C * K * 4, 4);
  bufs.in(bias, (size_t)C * 4, 4, false);
  bufs.in(state, held, e, false);
  bufs.in(lengths, (size_t)B * 4, 4, false);
  bufs.out(y, (size_t)B * N * C * e, e);
  bufs.out(state_out, held, e, false);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  ttt::Conv1dArgs a{};
  a.B = B, a.N = N, a.C = C, a.x = x, a.xs = x_stride, a.w = weight, a.bias = bias, a.state = state;
  a.lengths = lengths, a.y = y, a.state_out = state_out;
  return from_hip(ttt::conv1d_launch(dt == TTT_BF16, K, silu != 0, a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_step_conv1d(ttt_dtype dt, int B, int C, int K, int silu, const void* x,
                           long long x_stride, const float* weight, const float* bias,
                           const void* state, void* y, void* state_out, void* stream) {
  const ttt_status st = check_conv1d_sizes(dt, B, 1, C, K);
  if (st != TTT_OK) return st;
  if (silu != 0 && silu != 1) return TTT_ERR_INVALID;
  const size_t e = elem_size(dt), held = (size_t)B * (K - 1) * C * e;
  Buffers bufs;
  bufs.rows(x, B, x_stride, C, e);
  bufs.in(weight, (size_t)C * K * 4, 4);
  bufs.in(bias, (size_t)C * 4, 4, false);
  if (state != state_out) bufs.in(state, held, e);
  bufs.out(y, (size_t)B * C * e, e);
  bufs.out(state_out, held, e);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  ttt::Conv1dArgs a{};
  a.B = B, a.N = 1, a.C = C, a.x = x, a.xs = x_stride, a.w = weight, a.bias = bias, a.state = state;
  a.y = y, a.state_out = state_out;
  return from_hip(ttt::conv1d_step_launch(dt == TTT_BF16, K, silu != 0, a, static_cast<hipStream_t>(stream)));
}

size_t ttt_backward_conv1d_workspace(ttt_dtype dt, int B, int N, int C, int K) {
  if (check_conv1d_sizes(dt, B, N, C, K) != TTT_OK) return 0;
  return round_up(ttt::conv1d_bwd_workspace_bytes(dt == TTT_BF16, B, N, C, K), 256);
}

ttt_status ttt_backward_conv1d(ttt_dtype dt, int B, int N, int C, int K, int silu, const void* x,
                               long long x_stride, const float* weight, const float* bias,
                               const void* state, const int* lengths, const void* d_y, void* d_x,
                               float* d_weight, float* d_bias, void* d_state, void* workspace,
                               size_t workspace_bytes, void* stream) {
  ttt_status st = check_conv1d_sizes(dt, B, N, C, K);
  if (st != TTT_OK) return st;
  if ((silu != 0 && silu != 1) || (d_state && !state)) return TTT_ERR_INVALID;
  const size_t e = elem_size(dt), held = (size_t)B * (K - 1) * C * e, act = (size_t)B * N * C * e;
  Buffers bufs;
  bufs.rows(x, (long long)B * N, x_stride, C, e);
  bufs.in(weight, (size_t)C * K * 4, 4);
  bufs.in(bias, (size_t)C * 4, 4, false);
  bufs.in(state, held, e, false);
  bufs.in(lengths, (size_t)B * 4, 4, false);
  bufs.in(d_y, act, e);
  bufs.out(d_x, act, e);
  bufs.out(d_weight, (size_t)C * K * 4, 4);
  bufs.out(d_bias, (size_t)C * 4, 4, false);
  bufs.out(d_state, held, e, false);
  if (!bufs.ok()) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_backward_conv1d_workspace(dt, B, N, C, K));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  ttt::Conv1dArgs a{};
  a.B = B, a.N = N, a.C = C, a.x = x, a.xs = x_stride, a.w = weight, a.bias = bias, a.state = state;
  a.lengths = lengths, a.dy = d_y, a.dx = d_x, a.dw = d_weight, a.db = d_bias, a.dstate = d_state;
  a.partial = static_cast<float*>(workspace);
  return from_hip(ttt::conv1d_bwd_launch(dt == TTT_BF16, K, silu != 0, a, static_cast<hipStream_t>(stream)));
}

size_t ttt_forward_selective_scan_workspace(ttt_dtype dt, int B, int N, int C, int S, int G) {
  if (check_scan_sizes(dt, B, N, C, S, G) != TTT_OK) return 0;
  return round_up(ttt::scan_workspace_bytes(dt == TTT_BF16, B, N, C, S, G), 256);
}

ttt_status ttt_forward_selective_scan(ttt_dtype dt, int B, int N, int C, int S, int G, int softplus,
                                      const void* u, long long u_stride, const void* delta,
                                      long long delta_stride, const float* A, const void* Bm,
                                      long long b_stride, const void* Cm, long long c_stride,
                                      const float* D, const float* delta_bias, const void* z,
                                      long long z_stride, const float* h0, const int* lengths,
                                      void* y, float* h_out, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  ttt_status st = check_scan_sizes(dt, B, N, C, S, G);
  if (st != TTT_OK) return st;
  if (softplus != 0 && softplus != 1) return TTT_ERR_INVALID;
  ttt::ScanArgs a{};
  a.B = B, a.N = N, a.C = C, a.G = G, a.softplus = softplus, a.u = u, a.delta = delta, a.bm = Bm, a.cm = Cm, a.z = z;
  a.us = u_stride, a.ds = delta_stride, a.bs = b_stride, a.cs = c_stride, a.zs = z_stride;
  a.A = A, a.D = D, a.dbias = delta_bias, a.h0 = h0, a.lengths = lengths, a.y = y, a.h_out = h_out;
  const size_t held = (size_t)B * C * S * 4;
  Buffers bufs;
  add_scan_inputs(bufs, dt, B, N, S, a);
  bufs.in(h0, held, 4, false);
  bufs.out(y, (size_t)B * N * C * elem_size(dt), elem_size(dt));
  bufs.out(h_out, held, 4, false);
  if (!bufs.ok() || !dword_rows(a, dt)) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_forward_selective_scan_workspace(dt, B, N, C, S, G));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::scan_launch(dt == TTT_BF16, S, a, workspace, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_step_selective_scan(ttt_dtype dt, int B, int C, int S, int G, int softplus,
                                   const void* u, long long u_stride, const void* delta,
                                   long long delta_stride, const float* A, const void* Bm,
                                   long long b_stride, const void* Cm, long long c_stride,
                                   const float* D, const float* delta_bias, const void* z,
                                   long long z_stride, const float* h, void* y, float* h_out,
                                   void* stream) {
  const ttt_status st = check_scan_sizes(dt, B, 1, C, S, G);
  if (st != TTT_OK) return st;
  if (softplus != 0 && softplus != 1) return TTT_ERR_INVALID;
  ttt::ScanArgs a{};
  a.B = B, a.N = 1, a.C = C, a.G = G, a.softplus = softplus, a.u = u, a.delta = delta, a.bm = Bm, a.cm = Cm, a.z = z;
  a.us = u_stride, a.ds = delta_stride, a.bs = b_stride, a.cs = c_stride, a.zs = z_stride;
  a.A = A, a.D = D, a.dbias = delta_bias, a.h0 = h, a.y = y, a.h_out = h_out;
  const size_t held = (size_t)B * C * S * 4;
  Buffers bufs;
  add_scan_inputs(bufs, dt, B, 1, S, a);
  if (h != h_out) bufs.in(h, held, 4);
  bufs.out(h_out, held, 4);
  bufs.out(y, (size_t)B * C * elem_size(dt), elem_size(dt));
  if (!bufs.ok() || !dword_rows(a, dt)) return TTT_ERR_INVALID;
  return from_hip(ttt::scan_step_launch(dt == TTT_BF16, S, a, static_cast<hipStream_t>(stream)));
}

size_t ttt_backward_selective_scan_workspace(ttt_dtype dt, int B, int N, int C, int S, int G) {
  if (check_scan_sizes(dt, B, N, C, S, G) != TTT_OK) return 0;
  return round_up(ttt::scan_bwd_workspace_bytes(dt == TTT_BF16, B, N, C, S, G), 256);
}

ttt_status ttt_backward_selective_scan(ttt_dtype dt, int B, int N, int C, int S, int G, int softplus,
                                       const void* u, long long u_stride, const void* delta,
                                       long long delta_stride, const float* A, const void* Bm,
                                       long long b_stride, const void* Cm, long long c_stride,
                                       const float* D, const float* delta_bias, const void* z,
                                       long long z_stride, const float* h0, const int* lengths,
                                       const void* d_y, void* d_u, void* d_delta, float* d_A,
                                       void* d_B, void* d_C, float* d_D, float* d_delta_bias,
                                       void* d_z, float* d_h0, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  ttt_status st = check_scan_sizes(dt, B, N, C, S, G);
  if (st != TTT_OK) return st;
  if ((softplus != 0 && softplus != 1) || !z != !d_z) return TTT_ERR_INVALID;
  ttt::ScanArgs a{};
  a.B = B, a.N = N, a.C = C, a.G = G, a.softplus = softplus, a.u = u, a.delta = delta, a.bm = Bm, a.cm = Cm, a.z = z;
  a.us = u_stride, a.ds = delta_stride, a.bs = b_stride, a.cs = c_stride, a.zs = z_stride;
  a.A = A, a.D = D, a.dbias = delta_bias, a.h0 = h0, a.lengths = lengths, a.dy = d_y;
  a.du = d_u, a.ddelta = d_delta, a.dbm = d_B, a.dcm = d_C, a.dz = d_z, a.dA = d_A, a.dD = d_D;
  a.ddbias = d_delta_bias, a.dh0 = d_h0;
  const size_t e = elem_size(dt), held = (size_t)B * C * S * 4, act = (size_t)B * N * C * e;
  const size_t mat = (size_t)B * N * G * S * e;
  Buffers bufs;
  add_scan_inputs(bufs, dt, B, N, S, a);
  bufs.in(h0, held, 4, false);
  bufs.in(d_y, act, e);
  bufs.out(d_u, act, e);
  bufs.out(d_delta, act, e);
  bufs.out(d_z, act, e, false);
  bufs.out(d_B, mat, e);
  bufs.out(d_C, mat, e);
  bufs.out(d_A, (size_t)C * S * 4, 4);
  bufs.out(d_D, (size_t)C * 4, 4, false);
  bufs.out(d_delta_bias, (size_t)C * 4, 4, false);
  bufs.out(d_h0, held, 4, false);
  if (!bufs.ok() || !dword_rows(a, dt)) return TTT_ERR_INVALID;
  st = add_workspace(bufs, workspace, workspace_bytes, ttt_backward_selective_scan_workspace(dt, B, N, C, S, G));
  if (st != TTT_OK) return st;
  if (!bufs.ok()) return TTT_ERR_INVALID;
  return from_hip(ttt::scan_bwd_launch(dt == TTT_BF16, S, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
