// Dropout of an activation, added to a residual stream or not: y = residual + x keep / (1 - p). The gradient of x is the same
// of d_y. The mask comes from philox.hpp's counters, 8 channels of a row to one.
//
// A stream bound by HBM. Where rows are whole pieces of 8 channels and 16-byte aligned, a thread takes a piece and its
// number is its counter. Otherwise a wave takes 512 channels of a row: its lanes evaluate a
// counter each, and the masks go round, so that the loads and stores of single elements are of neighbours.
#include "internal.hpp"
#include "lm.hpp"
#include "philox.hpp"

namespace ttt {
namespace {

constexpr int kThreads = 256;

template <class T>
struct Piece8 {
  static constexpr int V = sizeof(T) == 2 ? 8 : 4;
  Raw<T, V> r[8 / V];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) r[i].load(p + i * V);
  }
  __device__ __forceinline__ void widen(float* v) const {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) r[i].widen(v + i * V);
  }
  static __device__ __forceinline__ void store(T* p, const float* v) {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) store_row<T, V>(p + i * V, v + i * V);
  }
};

// `per`: pieces of a row, 0 where the rows of x are back to back.
template <class T, bool ADD>
__global__ __launch_bounds__(kThreads) void dropout_pieces(const T* x, long long xs, const T* res, T* y, long long pieces,
                                                           unsigned per, Drop d) {
  const long long id = wide_block() * kThreads + threadIdx.x;
  if (id >= pieces) return;
  long long from = id * 8;
  if (per) {  // (fewer than 2^32 pieces then)
    const unsigned row = (unsigned)id / per;
    from = row * xs + ((unsigned)id - row * per) * 8;
  }
  Piece8<T> px, pr;
  px.load(x + from);
  if (ADD) pr.load(res + id * 8);
  Random8 u{};
  if (d.least) u = random8(d.rng[0], d.rng[1] + (unsigned long long)id);
  float v[8], r[8] = {};
  px.widen(v);
  if (ADD) pr.widen(r);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (u.kept(j, d.least) ? v[j] * d.scale : 0.f) + r[j];
  Piece8<T>::store(y + id * 8, v);
}

template <class T, bool ADD>
__global__ __launch_bounds__(kThreads) void dropout_rows(const T* x, long long xs, const T* res, T* y, int M, int C,
                                                         int parts, Drop d) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const long long id = wide_block() * (kThreads / 64) + wave;
  const long long row = id / parts;
  if (row >= M) return;
  const int c0 = (int)(id - row * parts) * 512;
  const T* px = x + row * xs + c0;
  const long long o = row * C + c0;
  T vx[8], vr[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int at = c0 + k * 64 + lane < C ? k * 64 + lane : 0;
    vx[k] = px[at];
    if (ADD) vr[k] = res[o + at];
  }
  RowMask<64, 8, 1> m;
  if (d.least)
    m.make(d.rng[0], d.rng[1] + (unsigned long long)row * (unsigned)((C + 7) / 8) + (unsigned)(c0 / 8), d.least, lane);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const bool keep = !d.least || m.kept(k, 0);
    const float v = (keep ? (float)vx[k] * d.scale : 0.f) + (ADD ? (float)vr[k] : 0.f);
    if (c0 + k * 64 + lane < C) y[o + k * 64 + lane] = (T)v;
  }
}

template <class T, bool ADD>
hipError_t launch(const DropoutArgs& a, hipStream_t st) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                       reinterpret_cast<uintptr_t>(a.y);
  const long long pieces = (long long)a.M * (a.C / 8);
  const bool flat = a.xs == a.C || a.M == 1;
  if (a.C % 8 == 0 && (flat || (a.xs * (int)sizeof(T) % 16 == 0 && pieces >> 32 == 0)) && (at & 15) == 0) {
    hipLaunchKernelGGL((dropout_pieces<T, ADD>), wide_grid((pieces + kThreads - 1) / kThreads), dim3(kThreads), 0, st,
                       (const T*)a.x, a.xs, (const T*)a.residual, (T*)a.y, pieces, flat ? 0u : (unsigned)a.C / 8, a.drop);
  } else {
    const int parts = (a.C + 511) / 512, per = kThreads / 64;
    hipLaunchKernelGGL((dropout_rows<T, ADD>), wide_grid(((long long)a.M * parts + per - 1) / per), dim3(kThreads), 0, st,
                       (const T*)a.x, a.xs, (const T*)a.residual, (T*)a.y, a.M, a.C, parts, a.drop);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t dropout_launch(bool bf16_io, const DropoutArgs& a, hipStream_t st) {
  return bf16_io ? (a.residual ? launch<bf16, true>(a, st) : launch<bf16, false>(a, st))
                 : (a.residual ? launch<float, true>(a, st) : launch<float, false>(a, st));
}

}  // namespace ttt
