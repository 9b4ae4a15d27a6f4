// Gated linear recurrence: forward, one token at a time, and backward. Per channel,
//   la = -scale softplus(lam) sigmoid(r),  a = exp(la),  m = sqrt(1 - a^2),  h = a h + m sigmoid(i) x,  y = h.
// Backward, with q_n = dy_n + a_{n+1} q_{n+1}:
//   dx = q m sig(i),  di = q m x sig(i) (1 - sig(i)),  t = q (a la h_{n-1} - a^2 (la / m) sig(i) x),
//   dr = t (1 - sig(r)),  dlam = sum t sig(lam) / softplus(lam),  dh0 = a_0 q_0.
// t is la times the gradient of la: m's derivative -a^2 / m is infinite where a is 1, but la / m goes to 0 there
// with the root of la.
//
// A thread walks a channel of a sequence from end to end.
#include "internal.hpp"
#include "lm.hpp"
#include "rowops.hpp"

namespace ttt {
namespace {

constexpr int kThreads = 64;
constexpr int kKept = 64;  // tokens between kept states

// 1 - exp(u) for u <= 0: by -u times a polynomial for u > -1/2 (within 1.1 * 2^-24 of it, found by Chebyshev's nodes), where the
// difference would lose bits; e is exp(u).
__device__ __forceinline__ float one_minus(float u, float e) {
  float p = 0.0011237150756642222f;
  p = fmaf(p, u, 0.008190003223717213f);
  p = fmaf(p, u, 0.04163024201989174f);
  p = fmaf(p, u, 0.16666245460510254f);
  p = fmaf(p, u, 0.4999998211860657f);
  p = fmaf(p, u, 1.f);
  return u > -0.5f ? -u * p : 1.f - e;
}

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

struct Gates {
  float gr, gi, la, a, w;  // sigmoid(r), sigmoid(i), log a, a, 1 - a^2
  __device__ __forceinline__ Gates(float r, float i, float k) {
    gr = sigmoid(r), gi = sigmoid(i);
    la = -k * gr;
    a = exp2_hw(kLog2e * la);
    w = one_minus(2.f * la, a * a);
  }
};

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

template <class T>
__global__ __launch_bounds__(kThreads) void recurrence_fwd(RecurrenceArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y, C = a.C;
  if (c >= C) return;
  const int n = length_of(a.lengths, b, a.N);
  const float k = a.scale * softplus(a.lam[c]);
  float h = a.h0 ? a.h0[(long long)b * C + c] : 0.f;
  float* states = a.states ? a.states + (long long)b * ((a.N + kKept - 1) / kKept) * C + c : nullptr;
  for (int t = 0; t < a.N; ++t) {
    if (states && t % kKept == 0) states[(long long)(t / kKept) * C] = h;
    const long long at = (long long)b * a.N + t;
    if (t < n) {
      const Gates g((float)((const T*)a.r)[at * a.rs + c], (float)((const T*)a.i)[at * a.is + c], k);
      h = fmaf(g.a, h, sqrtf(g.w) * g.gi * (float)((const T*)a.x)[at * a.xs + c]);
    }
    if (a.y) ((T*)a.y)[at * C + c] = (T)(t < n ? h : 0.f);
  }
  if (a.h_out) a.h_out[(long long)b * C + c] = h;
}

template <class T>
__global__ __launch_bounds__(kThreads) void recurrence_step(RecurrenceArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y, C = a.C;
  if (c >= C) return;
  const Gates g((float)((const T*)a.r)[b * a.rs + c], (float)((const T*)a.i)[b * a.is + c], a.scale * softplus(a.lam[c]));
  const long long at = (long long)b * C + c;
  const float h = fmaf(g.a, a.h0[at], sqrtf(g.w) * g.gi * (float)((const T*)a.x)[b * a.xs + c]);
  ((T*)a.y)[at] = (T)h;
  a.h_out[at] = h;
}

template <class T>
__global__ __launch_bounds__(kThreads) void recurrence_bwd(RecurrenceArgs a, float* before, float* part) {
  const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y, C = a.C;
  if (c >= C) return;
  const int n = length_of(a.lengths, b, a.N);
  const float k = a.scale * softplus(a.lam[c]);
  float h = a.h0 ? a.h0[(long long)b * C + c] : 0.f;
  for (int t = 0; t < n; ++t) {
    const long long at = (long long)b * a.N + t;
    before[at * C + c] = h;
    const Gates g((float)((const T*)a.r)[at * a.rs + c], (float)((const T*)a.i)[at * a.is + c], k);
    h = fmaf(g.a, h, sqrtf(g.w) * g.gi * (float)((const T*)a.x)[at * a.xs + c]);
  }
  float z = 0.f, sum = 0.f;  // a_{n+1} q_{n+1}; the sum of t
  for (int t = a.N - 1; t >= 0; --t) {
    const long long at = (long long)b * a.N + t;
    float dx = 0.f, dr = 0.f, di = 0.f;
    if (t < n) {
      const float x = (float)((const T*)a.x)[at * a.xs + c];
      const Gates g((float)((const T*)a.r)[at * a.rs + c], (float)((const T*)a.i)[at * a.is + c], k);
      const float q = (float)((const T*)a.dy)[at * C + c] + z, m = sqrtf(g.w);
      const float per = g.w == 0.f ? 0.f : g.la / m;
      const float l = q * (g.a * g.la * before[at * C + c] - g.a * g.a * per * g.gi * x);
      dx = q * m * g.gi;
      di = dx * x * (1.f - g.gi);
      dr = l * (1.f - g.gr);
      sum += l;
      z = g.a * q;
    }
    ((T*)a.dx)[at * C + c] = (T)dx;
    ((T*)a.dr)[at * C + c] = (T)dr;
    ((T*)a.di)[at * C + c] = (T)di;
  }
  part[(long long)b * C + c] = sum;
  if (a.dh0) a.dh0[(long long)b * C + c] = z;
}

// sigmoid(lam) / softplus(lam), 1 - exp(lam) / 2 and so on far below zero.
struct StoreDecayGrad {
  const float* lam;
  float* dlam;
  __device__ void operator()(int c, float s) const {
    const float l = lam[c];
    dlam[c] = s * (l < -20.f ? 1.f : 1.f / ((1.f + expf(-l)) * softplus(l)));
  }
};

dim3 grid_of(const RecurrenceArgs& a) { return dim3((unsigned)((a.C + kThreads - 1) / kThreads), (unsigned)a.B); }

}  // namespace

size_t recurrence_workspace_bytes(bool, int, int, int) { return 0; }

hipError_t recurrence_launch(bool bf16_io, const RecurrenceArgs& a, void*, hipStream_t st) {
  if (bf16_io) hipLaunchKernelGGL(recurrence_fwd<bf16>, grid_of(a), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL(recurrence_fwd<float>, grid_of(a), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t recurrence_step_launch(bool bf16_io, const RecurrenceArgs& a, hipStream_t st) {
  if (bf16_io) hipLaunchKernelGGL(recurrence_step<bf16>, grid_of(a), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL(recurrence_step<float>, grid_of(a), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

size_t recurrence_bwd_workspace_bytes(bool, int B, int N, int C, bool) { return ((size_t)B * N * C + (size_t)B * C) * 4; }

hipError_t recurrence_bwd_launch(bool bf16_io, const RecurrenceArgs& a, void* ws, hipStream_t st) {
  float* before = static_cast<float*>(ws);
  float* part = before + (size_t)a.B * a.N * a.C;
  if (bf16_io) hipLaunchKernelGGL(recurrence_bwd<bf16>, grid_of(a), dim3(kThreads), 0, st, a, before, part);
  else hipLaunchKernelGGL(recurrence_bwd<float>, grid_of(a), dim3(kThreads), 0, st, a, before, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return column_sum_launch(part, a.B, a.C, StoreDecayGrad{a.lam, a.dlam}, st);
}

}  // namespace ttt
