// Dropout of an activation, added to a residual stream or not: y = residual + x keep / (1 - p). The gradient of x is the same
// of d_y. The mask comes from philox.hpp's counters, 8 channels of a row to one.
//
// A stream bound by HBM: a thread takes the 8 channels of a counter, in 16-byte accesses at whatever alignment the rows have.
// 50176 x 384 in bf16 with a residual 18.5 us (6.2 TB/s, part of it from the cache behind L2), 50176 x 383 21.4; 12544 x 384
// 6.3 us; 1537 x 1001 in fp32 4.1, a launch and the bytes.
#include "internal.hpp"
#include "lm.hpp"
#include "pieces.hpp"

namespace ttt {
namespace {

constexpr int kThreads = 256;

// The 8 elements of a counter.
template <class T>
struct Eight {
  static constexpr int N = 8 / kPiece<T>;
  Piece<T> r[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].load(p + i * kPiece<T>);
  }
  __device__ __forceinline__ void widen(float* v) const {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].widen(v + i * kPiece<T>);
  }
  static __device__ __forceinline__ void store(T* p, const float* v) {
#pragma unroll
    for (int i = 0; i < N; ++i) Piece<T>::store(p + i * kPiece<T>, v + i * kPiece<T>);
  }
  // The last `count`, of 1 .. 7, to p.
  static __device__ __forceinline__ void store_last(T* p, const float* v, int count) {
    if constexpr (N == 1) {
      Piece<T>::store_last(p, v, count);
    } else {
#pragma unroll
      for (int j = 1; j < 8; ++j)
        if (j >= 8 - count) p[count - 8 + j] = v[j];
    }
  }
};

// `per`: counters of a row.
template <class T, bool ADD>
__global__ __launch_bounds__(kThreads) void dropout(const T* x, long long xs, const T* res, T* y, long long count, unsigned per,
                                                    int C, Drop d) {
  const long long id = wide_block() * kThreads + threadIdx.x;
  if (id >= count) return;
  long long row, at = id * 8, from = at;
  unsigned piece = 0;
  if (xs != C || C % 8 != 0) {  // (otherwise rows are one behind the other)
    if (count >> 32) row = id / per;
    else row = (unsigned)id / per;
    piece = (unsigned)(id - row * per);
    from = row * xs + (long long)piece * 8, at = row * C + (long long)piece * 8;
  }
  // The end of a row of another width is taken with its last 8 elements, where it has as many: the first `skip` are the counter's before.
  const int rest = C % 8;
  const bool whole = rest == 0 || piece < per - 1;
  const int skip = whole ? 0 : 8 - rest;
  float v[8] = {}, r[8] = {};
  Eight<T> px, pr;
  if (C >= 8) {
    px.load(x + from - skip);
    if (ADD) pr.load(res + at - skip);
  } else {
#pragma unroll
    for (int j = 1; j < 8; ++j)
      if (j >= skip) {
        v[j] = (float)x[from - skip + j];
        if (ADD) r[j] = (float)res[at - skip + j];
      }
  }
  uint32_t kept = 0xff;
  if (d.least) kept = random8(d.rng[0], d.rng[1] + (unsigned long long)id).mask(d.least) << skip;
  if (C >= 8) {
    px.widen(v);
    if (ADD) pr.widen(r);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = ((kept >> j) & 1 ? v[j] * d.scale : 0.f) + r[j];
  if (whole) Eight<T>::store(y + at, v);
  else Eight<T>::store_last(y + at, v, rest);
}

template <class T, bool ADD>
hipError_t launch(const DropoutArgs& a, hipStream_t st) {
  const unsigned per = ((unsigned)a.C + 7) / 8;
  const long long count = (long long)a.M * per;
  hipLaunchKernelGGL((dropout<T, ADD>), wide_grid((count + kThreads - 1) / kThreads), dim3(kThreads), 0, st, (const T*)a.x,
                     a.M == 1 ? a.C : a.xs, (const T*)a.residual, (T*)a.y, count, per, a.C, a.drop);
  return hipGetLastError();
}

}  // namespace

hipError_t dropout_launch(bool bf16_io, const DropoutArgs& a, hipStream_t st) {
  return bf16_io ? (a.residual ? launch<bf16, true>(a, st) : launch<bf16, false>(a, st))
                 : (a.residual ? launch<float, true>(a, st) : launch<float, false>(a, st));
}

}  // namespace ttt
