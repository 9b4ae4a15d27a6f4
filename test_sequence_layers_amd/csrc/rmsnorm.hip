// RMS norm over each head's D channels, forward and backward, with the residual's addition (and dropout of what is added)
// before it and, forward, an output in 8 bits after it.
//   s = residual + x keep / (1 - p),  y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   e4m3: q = y / scale,  scale = max |y| over a row or a group of its channels / 448
//   ds = dsum + rstd (g - xhat mean(g xhat)),  g = dy w,  xhat = s rstd;   dx = ds keep / (1 - p);   dw = sum dy xhat.
//
// A stream of rows, bound by HBM, laid out as layer norm's (normrows.hpp): a row is read once into the registers of L
// lanes, and the sum, the statistics, the maxima and every output come from there. Apart, the addition, the norm and
// the conversion would read and write the row two more times each.
#include "internal.hpp"
#include "lm.hpp"
#include "normrows.hpp"
#include "philox.hpp"

namespace ttt {
namespace {

// rstd of a row, times *back; v is scaled by 1 / *back where its squares overflow (from 2^60 or so on: the largest squares
// are 2^96 then, and eps is nothing beside them), so that such rows are normed like others. An infinite or NaN entry makes its row
// NaN at least where the entry is.
template <int L, int K, int V>
__device__ __forceinline__ float inverse_rms(float* v, int D, float eps, float (*red)[16], float* back) {
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < K * V; ++j) q = fmaf(v[j], v[j], q);
  q = row_sum<L>(q, red, 0);
  *back = 1.f;
  const bool over = !(q < __builtin_inff());
  if (__ballot(over)) {  // (rows of more than a wave: the same for all of it)
    const float down = over ? 0x1p-80f : 1.f;
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < K * V; ++j) {
      v[j] *= down;
      t = fmaf(v[j], v[j], t);
    }
    q = row_sum<L>(t, red, 1);
    eps = over ? 0.f : eps;
    *back = down;
  }
  return rcp_hw(sqrtf(fmaf(q, rcp_hw((float)D), eps)));
}

// v -> residual + v keep scale (v's own values where there is no residual), the values before they are rounded.
template <int L, int K, int V>
__device__ __forceinline__ void drop_row(float* v, const Drop& d, long long row, int D, int lane) {
  RowMask<L, K, V> m;
  m.make(d.rng[0], d.rng[1] + (unsigned long long)row * (unsigned)((D + 7) / 8), d.least, lane);
#pragma unroll
  for (int k = 0; k < K; ++k)
    for (int i = 0; i < V; ++i) v[k * V + i] = m.kept(k, i) ? v[k * V + i] * d.scale : 0.f;
}

// Largest value over aligned groups of L lanes (runtime L, a power of two).
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int L) {
  auto other = [](uint32_t a, int which) {
    const int x = (int)a;
    return (uint32_t)(which == 1 ? __builtin_amdgcn_update_dpp(0, x, kDppXor1, 0xf, 0xf, true)
                      : which == 2 ? __builtin_amdgcn_update_dpp(0, x, kDppXor2, 0xf, 0xf, true)
                      : which == 4 ? __builtin_amdgcn_update_dpp(0, x, kDppMirror8, 0xf, 0xf, true)
                                   : __builtin_amdgcn_update_dpp(0, x, kDppMirror16, 0xf, 0xf, true));
  };
  if (L >= 2) v = max(v, other(v, 1));
  if (L >= 4) v = max(v, other(v, 2));
  if (L >= 8) v = max(v, other(v, 4));
  if (L >= 16) v = max(v, other(v, 8));
  if (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  if (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  return v;
}

// Four e4m3 of four fp32, rounded to nearest even; values are within +-448 (1 + 2^-22) or NaN.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* v) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(to_e4m3(v[0], v[1], v[2], v[3]), to_e4m3(v[4], v[5], v[6], v[7]));
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p) = to_e4m3(v[0], v[1], v[2], v[3]);
  } else {
    p[0] = (uint8_t)to_e4m3(v[0], 0.f, 0.f, 0.f);
  }
}

constexpr float kE4m3Most = 448.f;
constexpr float kLeastMax = 0x1p-100f;  // a smaller maximum's inverse could be infinite; such values are zeros in 8 bits

template <class T, int L, int K, int V, bool ADD, bool E4M3>
__global__ __launch_bounds__(threads_of<L>) void rmsnorm_fwd(const T* __restrict__ x, long long xs, const T* res,
                                                             const float* __restrict__ w, T* sum, void* __restrict__ y,
                                                             float* __restrict__ scales, int rows, int H, int D,
                                                             int group, float eps, Drop drop) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x % L;
  const long long row = wide_block() * (threads_of<L> / L) + threadIdx.x / L;
  if (row >= rows) return;  // (whole groups; for L > 64 the whole workgroup)
  const int m = (int)(row / H), h = (int)(row - (long long)m * H);
  Row<T, L, K, V> rx, rr;
  rx.load(x + (long long)m * xs + (long long)h * D, lane, D);
  if (ADD) rr.load(res + row * D, lane, D);
  float v[K * V];
  rx.widen(v, lane, D);
  if (ADD) {
    if (drop.least) drop_row<L, K, V>(v, drop, row, D, lane);
    float r[K * V];
    rr.widen(r, lane, D);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      for (int i = 0; i < V; ++i) v[k * V + i] += r[k * V + i];
      if (at < D) store_row<T, V>(sum + row * D + at, v + k * V);
    }
  }
  float back;
  const float rstd = inverse_rms<L, K, V>(v, D, eps, red, &back);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int at = (k * L + lane) * V;
    float wv[V];
    load_params<V>(w + (long long)h * D + (at < D ? at : 0), wv);
    for (int i = 0; i < V; ++i) v[k * V + i] *= rstd * wv[i];
  }
  if constexpr (!E4M3) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      if (at < D) store_row<T, V>((T*)y + row * D + at, v + k * V);
    }
  } else {
    // Maxima of the absolute values' bits: as numbers they are in the same order, and a NaN is above all.
    uint32_t most[K], all = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      most[k] = 0;
      if ((k * L + lane) * V < D)
        for (int i = 0; i < V; ++i) most[k] = max(most[k], __float_as_uint(v[k * V + i]) & 0x7fffffffu);
      all = max(all, most[k]);
    }
    if (group == D) {
      all = lanes_max(all, L < 64 ? L : 64);
      if constexpr (L > 64) {
        __shared__ uint32_t tops[16];
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = all;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < L / 64; ++i) all = max(all, tops[i]);
      }
    }
    const int share = group / V;  // lanes of a group, where it is less than the row
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      float top = __uint_as_float(group == D ? all : lanes_max(most[k], share));
      top = top < kLeastMax ? kLeastMax : top;
      const float inv = kE4m3Most / top;
      if (at < D) {
        for (int i = 0; i < V; ++i) v[k * V + i] *= inv;
        store_e4m3<V>((uint8_t*)y + row * D + at, v + k * V);
        if (group == D ? at == 0 : (lane & (share - 1)) == 0) scales[(row * D + at) / group] = top / kE4m3Most;
      }
    }
  }
}

// Workgroup (bx, by): as in layer norm's backward pass, R tokens at a time of the HB heads from by HB on. Partial row bx: dw (H D).
template <class T, int L, int K, int V, bool ADD>
__global__ __launch_bounds__(bwd_threads(L, K* V)) void rmsnorm_bwd(const T* __restrict__ s, long long ss,
                                                                    const float* __restrict__ w,
                                                                    const T* __restrict__ dy, const T* dsum, T* ds,
                                                                    T* __restrict__ dx, float* __restrict__ part, int M,
                                                                    int H, int D, int HB, int R, float eps, Drop drop) {
  constexpr int LKV = L * K * V;
  constexpr bool kRoom = L <= 256;  // (as in layer norm's backward pass)
  __shared__ float red[4][16];
  __shared__ float join[L <= 64 ? bwd_threads(L, K * V) * K * V : 1];
  const int lane = threadIdx.x % L, g = threadIdx.x / L;
  const int r = g / HB, hg = blockIdx.y * HB + g % HB, h = min(hg, H - 1);
  const bool live = r < R && hg < H;
  const float inv_d = rcp_hw((float)D);
  float wv[K * V], aw[K * V] = {};
  auto weights = [&]() {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      load_params<V>(w + (long long)h * D + (at < D ? at : 0), wv + k * V);
    }
  };
  if (kRoom) weights();
  Row<T, L, K, V> rx, rd, rr;
  auto fetch = [&](long long m) {  // (past the last token: the last again)
    const long long t = m < M ? m : M - 1;
    rx.load(s + t * ss + (long long)h * D, lane, D);
    rd.load(dy + (t * H + h) * D, lane, D);
    if (ADD) rr.load(dsum + (t * H + h) * D, lane, D);
  };
  const long long step = (long long)gridDim.x * R;
  if (kRoom) fetch((long long)blockIdx.x * R + r);
  for (long long m0 = (long long)blockIdx.x * R; m0 < M; m0 += step) {
    const long long m = m0 + r;
    const bool in = live && m < M;
    float v[K * V], d[K * V], e[K * V];
    if (!kRoom) fetch(m);
    rx.widen(v, lane, D);
    rd.widen(d, lane, D, in);
    if (ADD) rr.widen(e, lane, D, in);
    if (kRoom) fetch(m + step);
    float back;
    const float rstd = inverse_rms<L, K, V>(v, D, eps, red, &back);
    if (!kRoom) weights();
    float s2 = 0.f;
#pragma unroll
    for (int j = 0; j < K * V; ++j) {
      v[j] *= rstd;  // xhat
      aw[j] += in ? d[j] * v[j] : 0.f;
      d[j] *= wv[j];  // g
      s2 = fmaf(d[j], v[j], s2);
    }
    s2 = row_sum<L>(s2, red, 2) * inv_d;
    const float outer = rstd * back;
#pragma unroll
    for (int j = 0; j < K * V; ++j) d[j] = outer * (d[j] - v[j] * s2) + (ADD ? e[j] : 0.f);
    const long long o = (m * H + h) * D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      if (in && at < D) store_row<T, V>(ds + o + at, d + k * V);
    }
    if (dx) {
      if (drop.least) drop_row<L, K, V>(d, drop, m, D, lane);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int at = (k * L + lane) * V;
        if (in && at < D) store_row<T, V>(dx + o + at, d + k * V);
      }
    }
  }
  const long long W = (long long)H * D;
  float* row = part + (long long)blockIdx.x * W;
  if constexpr (L > 64) {  // one group: its registers are the workgroup's sums
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int i = 0; i < V; ++i) {
        const int at = (k * L + lane) * V + i;
        if (at < D) row[(long long)h * D + at] = aw[k * V + i];
      }
  } else {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int i = 0; i < V; ++i) join[g * LKV + (k * L + lane) * V + i] = aw[k * V + i];
    __syncthreads();
    for (int t = threadIdx.x; t < HB * D; t += blockDim.x) {
      const int hh = t / D, at = t - hh * D;
      if (blockIdx.y * HB + hh >= H) break;
      float sum = 0.f;
      for (int q = 0; q < R; ++q) sum += join[(q * HB + hh) * LKV + at];
      row[(long long)(blockIdx.y * HB + hh) * D + at] = sum;
    }
  }
}

struct StoreWeightGrad {
  float* dw;
  __device__ void operator()(int col, float s) const { dw[col] = s; }
};

struct FwdCall {
  const RmsNormArgs& a;
  hipStream_t st;
  template <class T, int L, int K, int V>
  hipError_t run() const {
    return a.scales ? (a.residual ? go<T, L, K, V, true, true>() : go<T, L, K, V, false, true>())
                    : (a.residual ? go<T, L, K, V, true, false>() : go<T, L, K, V, false, false>());
  }
  template <class T, int L, int K, int V, bool ADD, bool E4M3>
  hipError_t go() const {
    constexpr int G = threads_of<L> / L;
    const int rows = a.M * a.H;
    hipLaunchKernelGGL((rmsnorm_fwd<T, L, K, V, ADD, E4M3>), wide_grid(((long long)rows + G - 1) / G), dim3(threads_of<L>), 0,
                       st, (const T*)a.x, a.xs, (const T*)a.residual, a.w, (T*)a.sum, a.y, a.scales, rows, a.H, a.D,
                       a.group, a.eps, a.drop);
    return hipGetLastError();
  }
};

struct BwdCall {
  const RmsNormArgs& a;
  BwdPlan p;
  hipStream_t st;
  template <class T, int L, int K, int V>
  hipError_t run() const {
    return a.dsum ? go<T, L, K, V, true>() : go<T, L, K, V, false>();
  }
  template <class T, int L, int K, int V, bool ADD>
  hipError_t go() const {
    const int threads = L <= 64 ? (p.HB * p.R * L + 63) / 64 * 64 : L;
    hipLaunchKernelGGL((rmsnorm_bwd<T, L, K, V, ADD>), dim3((unsigned)p.P, (unsigned)p.gy), dim3(threads), 0, st,
                       (const T*)a.x, a.xs, a.w, (const T*)a.dy, (const T*)a.dsum, (T*)a.ds, (T*)a.dx, a.partial, a.M,
                       a.H, a.D, p.HB, p.R, a.eps, a.drop);
    return hipGetLastError();
  }
};

}  // namespace

bool rmsnorm_vector(bool bf16_io, const RmsNormArgs& a) {
  const void* all[] = {a.x, a.residual, a.w, a.sum, a.dy, a.dsum, a.ds, a.dx};
  if (!vector_rows(bf16_io, a.D, a.xs)) return false;
  for (const void* p : all)
    if (!aligned16(p)) return false;
  const uintptr_t y = reinterpret_cast<uintptr_t>(a.y);  // in 8 bits an access is a byte for each element
  return (y & (a.scales ? (bf16_io ? 7u : 3u) : 15u)) == 0;
}

hipError_t rmsnorm_launch(bool bf16_io, const RmsNormArgs& a, hipStream_t st) {
  return with_shape(bf16_io, shape_of(bf16_io, rmsnorm_vector(bf16_io, a), a.D), FwdCall{a, st});
}

size_t rmsnorm_bwd_workspace_bytes(bool bf16_io, int M, int H, int D) {
  long long P = bwd_plan(shape_of(bf16_io, false, D), M, H).P;
  if (vector_rows(bf16_io, D, 0)) P = std::max(P, bwd_plan(shape_of(bf16_io, true, D), M, H).P);
  return (size_t)P * H * D * sizeof(float);
}

hipError_t rmsnorm_bwd_launch(bool bf16_io, const RmsNormArgs& a, hipStream_t st) {
  const Shape s = shape_of(bf16_io, rmsnorm_vector(bf16_io, a), a.D);
  const BwdPlan p = bwd_plan(s, a.M, a.H);
  const hipError_t e = with_shape(bf16_io, s, BwdCall{a, p, st});
  if (e != hipSuccess) return e;
  return column_sum_launch(a.partial, p.P, a.H * a.D, StoreWeightGrad{a.dw}, st);
}

}  // namespace ttt
