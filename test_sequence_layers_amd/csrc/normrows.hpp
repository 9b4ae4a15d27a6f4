// What the kernels of norms over rows share (layernorm.hip, rmsnorm.hip): a row of D channels held by L lanes, sums over
// it, and how calls are cut up.
#pragma once

#include <algorithm>

#include "rowops.hpp"

namespace ttt {
namespace {

constexpr int kThreads = 256;  // of a workgroup of several rows; a wide row has L threads to itself
template <int L>
constexpr int threads_of = L <= 64 ? kThreads : L;
// The backward pass: more rows to a workgroup where a lane holds few elements, so that fewer partial rows
// are written for as many waves (32768 x 12 x 64, bf16: 30.2 us, against 36.1 with 256 threads).
constexpr int bwd_threads(int L, int KV) { return L > 64 ? L : KV <= 8 ? 1024 : kThreads; }

// Sum over a row's L lanes; a row of more than a wave over its waves through LDS, `slot` going through
// 0 .. 3 with consecutive sums so that one barrier each is enough.
template <int L>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot) {
  if constexpr (L <= 64) {
    return lanes_sum<L>(v);
  } else {
    v = lanes_sum<64>(v);
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < L / 64; ++i) s += red[slot][i];
    return s;
  }
}

// One row: element (k L + lane) V + i is v[k V + i]. Past D the row's first elements are loaded again,
// and made `past` when they are used.
template <class T, int L, int K, int V>
struct Row {
  Raw<T, V> r[K];
  __device__ __forceinline__ void load(const T* p, int lane, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      r[k].load(p + (at < D ? at : 0));
    }
  }
  __device__ __forceinline__ void widen(float* v, int lane, int D, bool in = true, float past = 0.f) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r[k].widen(v + k * V);
      const bool ok = in && (k * L + lane) * V < D;
      for (int i = 0; i < V; ++i) v[k * V + i] = ok ? v[k * V + i] : past;
    }
  }
};

// How a row of D channels is spread over lanes: L lanes, K accesses of V elements each, at most 24 elements
// a lane (the backward pass holds five of such a set). A wave as far as that goes, since sums over more
// waves take a barrier each.
struct Shape {
  int L, K, V;
};
inline Shape shape_of(bool bf, bool vec, int D) {
  const int V = vec ? (bf ? 8 : 4) : 1;
  const int n = (D + V - 1) / V;  // accesses
  if (!vec) {
    if (n <= 64) return {64, 1, 1};
    if (n <= 256) return {64, 4, 1};
    if (n <= 1024) return {64, 16, 1};
    return n <= 4096 ? Shape{256, 16, 1} : Shape{1024, 16, 1};
  }
  for (int L = 8; L <= 64; L *= 2)
    if (n <= L) return {L, 1, V};
  if (n <= 128) return {64, 2, V};
  if (bf) {
    if (n <= 192) return {64, 3, V};
    if (n <= 512) return {256, n <= 256 ? 1 : 2, V};
    return {1024, n <= 1024 ? 1 : 2, V};
  }
  if (n <= 256) return {64, 4, V};
  if (n <= 1024) return {256, n <= 512 ? 2 : 4, V};
  return {1024, n <= 2048 ? 2 : 4, V};
}

// Calls f.run<T, L, K, V>() for the shape; every shape shape_of returns of 16-byte pieces is listed in with_pieces, with_shape has all.
template <class F>
hipError_t with_pieces(bool bf, Shape s, const F& f) {
#define TTT_LN(T, l, k, v) \
  if (s.L == l && s.K == k && s.V == v) return f.template run<T, l, k, v>();
  if (bf) {
    TTT_LN(bf16, 8, 1, 8) TTT_LN(bf16, 16, 1, 8) TTT_LN(bf16, 32, 1, 8) TTT_LN(bf16, 64, 1, 8)
    TTT_LN(bf16, 64, 2, 8) TTT_LN(bf16, 64, 3, 8) TTT_LN(bf16, 256, 1, 8) TTT_LN(bf16, 256, 2, 8)
    TTT_LN(bf16, 1024, 1, 8) TTT_LN(bf16, 1024, 2, 8)
  } else {
    TTT_LN(float, 8, 1, 4) TTT_LN(float, 16, 1, 4) TTT_LN(float, 32, 1, 4) TTT_LN(float, 64, 1, 4)
    TTT_LN(float, 64, 2, 4) TTT_LN(float, 64, 4, 4) TTT_LN(float, 256, 2, 4) TTT_LN(float, 256, 4, 4)
    TTT_LN(float, 1024, 2, 4) TTT_LN(float, 1024, 4, 4)
  }
  return hipErrorInvalidValue;
}
template <class F>
hipError_t with_shape(bool bf, Shape s, const F& f) {
#define TTT_LN_SCALAR(T) \
  TTT_LN(T, 64, 1, 1) TTT_LN(T, 64, 4, 1) TTT_LN(T, 64, 16, 1) TTT_LN(T, 256, 16, 1) TTT_LN(T, 1024, 16, 1)
  if (s.V > 1) return with_pieces(bf, s, f);
  if (bf) {
    TTT_LN_SCALAR(bf16)
  } else {
    TTT_LN_SCALAR(float)
  }
#undef TTT_LN_SCALAR
#undef TTT_LN
  return hipErrorInvalidValue;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 16-byte accesses need whole vectors per row and aligned rows.
inline bool vector_rows(bool bf, int D, long long xs) {
  const int V = bf ? 8 : 4;
  return D % V == 0 && xs % V == 0;
}

// The backward's grid: heads per workgroup, tokens at a time, workgroups along the tokens. It goes by the shape, so
// the 16-byte path and the other have different ones, and the workspace is sized for the larger.
struct BwdPlan {
  int HB, R, gy;
  long long P;
};
constexpr long long kTurns = 2048;
inline BwdPlan bwd_plan(Shape s, int M, int H) {
  const int threads = bwd_threads(s.L, s.K * s.V), groups = s.L <= 64 ? threads / s.L : 1;
  BwdPlan p;
  p.HB = H < groups ? H : groups;
  p.R = groups / p.HB;
  p.gy = (H + p.HB - 1) / p.HB;
  p.P = ((long long)M + p.R - 1) / p.R;
  // Workgroups: four waves per SIMD of 256 CUs with 1024 threads each, two with fewer (8192 x 4096: 50.5 us
  // with 512 workgroups, 55.8 with 768, 63 with 1024; 65536 x 768: 66.6, 63.7 and 67.1).
  // More where a group would walk further than kTurns rows, whose sums are one after the other: 32768 times 0.77 came
  // out off by 6770 times 2^-24, 16 times 2048 by 253.
  const long long wgs = threads >= 1024 ? 256 : 512;
  const long long most = std::max({1ll, wgs / p.gy, (p.P + kTurns - 1) / kTurns});
  if (p.P > most) {  // as many turns each, up to one
    const long long turns = (p.P + most - 1) / most;
    p.P = (p.P + turns - 1) / turns;
  }
  return p;
}

}  // namespace
}  // namespace ttt
