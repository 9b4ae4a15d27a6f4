// Layer norm over each head's D channels, forward and backward: a block is Norm -> layer -> residual
// (ViT^3 review on techloop.online, "TTT Block" section).
//   y = xhat w + b,  xhat = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy w;   dw = sum dy xhat,   db = sum dy.
//
// A stream of rows, bound by HBM: each row is read once into registers by a group of L lanes (8 lanes
// for a head of 64 bf16 channels, a wave, or a workgroup of 256 threads for wide rows), the
// statistics are taken there in two passes over the registers (the mean, then the centred squares:
// no cancellation; for the mean see RowX), and the result is written from them. The backward pass recomputes the
// statistics, since it has to read x anyway; each group keeps the same channels over the rows it
// walks, so that dw and db stay in registers until its last row; a workgroup's groups are joined in
// LDS, and a second launch sums the workgroups' partial rows in a fixed order. bf16: forward of 32768 x 12
// heads x 64 18.9 us (101 MB at 5.3 TB/s, the rate of a large copy), of 65536 x 768 34.7 us; backward of 65536 x
// 768 66.6 us (302 MB at 4.5 TB/s), of 12544 x 384 14.7 us, where the start and end of the two launches are
// most of it.
#include "internal.hpp"
#include "normrows.hpp"
#include "seq.hpp"

namespace ttt {
namespace {

// A row of x. In fp32 its first element comes along: the mean is taken of what the elements differ from it, so that a
// row far from zero loses what 24 bits of its differences lose and not of its values, and a constant row is centred to
// zeros (1e5 + N(0, 1): y off by 1e-2 without, 1e-6 with it; 1537 x 1001 backward 13.8 us with and without). In bf16 a row so
// far from zero for its spread has neighbouring values, and their sums are exact.
template <class T, int L, int K, int V>
struct RowX : Row<T, L, K, V> {
  static constexpr bool kFirst = sizeof(T) == 4;
  float first;
  __device__ __forceinline__ void load(const T* p, int lane, int D) {
    first = kFirst ? (float)p[0] : 0.f;
    Row<T, L, K, V>::load(p, lane, D);
  }
  // Row::widen, with the first element past D, which single elements are there already.
  __device__ __forceinline__ void widen(float* v, int lane, int D) const {
    if constexpr (kFirst && V == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) this->r[k].widen(v + k);
    } else {
      Row<T, L, K, V>::widen(v, lane, D, true, first);
    }
  }
};

// v -> v - mean (zero past D); returns rstd. With a first element the mean is the sum of two numbers, hi + lo, since
// as one it would be off by half a step of it.
template <bool FIRST, int L, int K, int V>
__device__ __forceinline__ float centre(float* v, float first, int lane, int D, float eps, float (*red)[16]) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < K * V; ++j) s += FIRST ? v[j] - first : v[j];
  const float mean = row_sum<L>(s, red, 0) / (float)D;
  const float hi = FIRST ? first + mean : mean, lo = FIRST ? (first - hi) + mean : 0.f;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    for (int i = 0; i < V; ++i) {
      float& x = v[k * V + i];
      x = (k * L + lane) * V < D ? (FIRST ? (x - hi) - lo : x - hi) : 0.f;
      q = fmaf(x, x, q);
    }
  return rcp_hw(sqrtf(fmaf(row_sum<L>(q, red, 1), rcp_hw((float)D), eps)));
}

template <class T, int L, int K, int V>
__global__ __launch_bounds__(threads_of<L>) void layernorm_fwd(const T* __restrict__ x, long long xs,
                                                               const float* __restrict__ w,
                                                               const float* __restrict__ b, T* __restrict__ y,
                                                               int rows, int H, int D, float eps) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x % L;
  const long long row = wide_block() * (threads_of<L> / L) + threadIdx.x / L;
  if (row >= rows) return;  // (whole groups; for L > 64 the whole workgroup)
  const int m = (int)(row / H), h = (int)(row - (long long)m * H);
  RowX<T, L, K, V> raw;
  raw.load(x + (long long)m * xs + (long long)h * D, lane, D);
  float v[K * V];
  raw.widen(v, lane, D);
  const float rstd = centre<raw.kFirst, L, K, V>(v, raw.first, lane, D, eps, red);
  T* py = y + row * D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int at = (k * L + lane) * V;
    if (at < D) {
      float wv[V], bv[V] = {};
      load_params<V>(w + (long long)h * D + at, wv);
      if (b) load_params<V>(b + (long long)h * D + at, bv);
      for (int i = 0; i < V; ++i) wv[i] = fmaf(v[k * V + i] * rstd, wv[i], bv[i]);
      store_row<T, V>(py + at, wv);
    }
  }
}

// Workgroup (bx, by): R tokens at a time of the HB heads from by HB on, tokens bx R + r, + gridDim.x R, ...
// Group g of L lanes has token r = g / HB and head g % HB; the next token's row is loaded while this one's
// is worked on. Partial row bx: [dw (H D), db (H D)].
template <class T, int L, int K, int V>
__global__ __launch_bounds__(bwd_threads(L, K* V)) void layernorm_bwd(const T* __restrict__ x, long long xs,
                                                               const float* __restrict__ w,
                                                               const T* __restrict__ dy, T* __restrict__ dx,
                                                               float* __restrict__ part, int M, int H, int D,
                                                               int HB, int R, float eps) {
  constexpr int LKV = L * K * V;
  // A workgroup of 1024 threads has 128 registers a lane: there the weights are read again for each row,
  // and rows are not loaded ahead. It is too few all the same for the widest rows, whose accumulators are partly
  // held in memory: 84 (fp32) and 73 registers of single elements, from 4097 channels on that are not whole
  // 16-byte pieces, 20 and 11 of aligned rows wider than 8192.
  constexpr bool kRoom = L <= 256;
  __shared__ float red[4][16];
  __shared__ float join[L <= 64 ? bwd_threads(L, K * V) * K * V : 1];
  const int lane = threadIdx.x % L, g = threadIdx.x / L;
  const int r = g / HB, hg = blockIdx.y * HB + g % HB, h = min(hg, H - 1);
  const bool live = r < R && hg < H;
  const float inv_d = rcp_hw((float)D);
  float wv[K * V], aw[K * V] = {}, ab[K * V] = {};
  auto weights = [&]() {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      load_params<V>(w + (long long)h * D + (at < D ? at : 0), wv + k * V);
    }
  };
  if (kRoom) weights();
  RowX<T, L, K, V> rx;
  Row<T, L, K, V> rd;
  auto fetch = [&](long long m) {  // (past the last token: the last again)
    const long long t = m < M ? m : M - 1;
    rx.load(x + t * xs + (long long)h * D, lane, D);
    rd.load(dy + (t * H + h) * D, lane, D);
  };
  const long long step = (long long)gridDim.x * R;
  if (kRoom) fetch((long long)blockIdx.x * R + r);
  for (long long m0 = (long long)blockIdx.x * R; m0 < M; m0 += step) {
    const long long m = m0 + r;
    const bool in = live && m < M;
    float v[K * V], d[K * V];
    if (!kRoom) fetch(m);
    rx.widen(v, lane, D);
    rd.widen(d, lane, D, in);
    const float first = rx.first;
    if (kRoom) fetch(m + step);
    const float rstd = centre<rx.kFirst, L, K, V>(v, first, lane, D, eps, red);
    if (!kRoom) weights();
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < K * V; ++j) {
      v[j] *= rstd;  // xhat
      ab[j] += d[j];
      aw[j] += in ? d[j] * v[j] : 0.f;
      d[j] *= wv[j];  // g
      s1 += d[j];
      s2 = fmaf(d[j], v[j], s2);
    }
    s1 = row_sum<L>(s1, red, 2) * inv_d;
    s2 = row_sum<L>(s2, red, 3) * inv_d;
    T* o = dx + (m * H + h) * D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (k * L + lane) * V;
      float ov[V];
      for (int i = 0; i < V; ++i) ov[i] = rstd * (d[k * V + i] - s1 - v[k * V + i] * s2);
      if (in && at < D) store_row<T, V>(o + at, ov);
    }
  }
  const long long W = (long long)H * D;
  float* row = part + (long long)blockIdx.x * 2 * W;
  if constexpr (L > 64) {  // one group: its registers are the workgroup's sums
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int i = 0; i < V; ++i) {
        const int at = (k * L + lane) * V + i;
        if (at < D) {
          row[(long long)h * D + at] = aw[k * V + i];
          row[W + (long long)h * D + at] = ab[k * V + i];
        }
      }
  } else {
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
        for (int i = 0; i < V; ++i) join[g * LKV + (k * L + lane) * V + i] = which ? ab[k * V + i] : aw[k * V + i];
      __syncthreads();
      for (int t = threadIdx.x; t < HB * D; t += blockDim.x) {
        const int hh = t / D, at = t - hh * D;
        if (blockIdx.y * HB + hh >= H) break;
        float s = 0.f;
        for (int q = 0; q < R; ++q) s += join[(q * HB + hh) * LKV + at];
        row[which * W + (long long)(blockIdx.y * HB + hh) * D + at] = s;
      }
    }
  }
}

struct StoreNormGrads {
  float *dw, *db;
  int W;
  __device__ void operator()(int col, float s) const {
    if (col < W) dw[col] = s;
    else if (db) db[col - W] = s;
  }
};

struct FwdCall {
  const void* x;
  long long xs;
  const float *w, *b;
  void* y;
  int M, H, D;
  float eps;
  hipStream_t st;
  template <class T, int L, int K, int V>
  hipError_t run() const {
    constexpr int G = threads_of<L> / L;
    const int rows = M * H;
    hipLaunchKernelGGL((layernorm_fwd<T, L, K, V>), wide_grid(((long long)rows + G - 1) / G), dim3(threads_of<L>), 0, st,
                       (const T*)x, xs, w, b, (T*)y, rows, H, D, eps);
    return hipGetLastError();
  }
};

struct BwdCall {
  const void* x;
  long long xs;
  const float* w;
  const void* dy;
  void* dx;
  float* part;
  int M, H, D;
  float eps;
  BwdPlan p;
  hipStream_t st;
  template <class T, int L, int K, int V>
  hipError_t run() const {
    const int threads = L <= 64 ? (p.HB * p.R * L + 63) / 64 * 64 : L;
    hipLaunchKernelGGL((layernorm_bwd<T, L, K, V>), dim3((unsigned)p.P, (unsigned)p.gy), dim3(threads), 0, st,
                       (const T*)x, xs, w, (const T*)dy, (T*)dx, part, M, H, D, p.HB, p.R, eps);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t layernorm_launch(bool bf16_io, int M, int H, int D, float eps, const void* x, long long xs,
                            const float* w, const float* b, void* y, hipStream_t st) {
  const bool vec = vector_rows(bf16_io, D, xs) && aligned16(x) && aligned16(w) && aligned16(b) && aligned16(y);
  return with_shape(bf16_io, shape_of(bf16_io, vec, D), FwdCall{x, xs, w, b, y, M, H, D, eps, st});
}

size_t layernorm_bwd_workspace_bytes(bool bf16_io, int M, int H, int D) {
  long long P = bwd_plan(shape_of(bf16_io, false, D), M, H).P;
  if (vector_rows(bf16_io, D, 0)) {
    const long long pv = bwd_plan(shape_of(bf16_io, true, D), M, H).P;
    if (pv > P) P = pv;
  }
  return (size_t)P * 2 * H * D * sizeof(float);
}

hipError_t layernorm_bwd_launch(bool bf16_io, int M, int H, int D, float eps, const void* x,
                                long long xs, const float* w, const void* dy, void* dx, float* dw,
                                float* db, void* ws, hipStream_t st) {
  const bool vec = vector_rows(bf16_io, D, xs) && aligned16(x) && aligned16(w) && aligned16(dy) && aligned16(dx);
  const Shape s = shape_of(bf16_io, vec, D);
  const BwdPlan p = bwd_plan(s, M, H);
  float* part = static_cast<float*>(ws);
  const hipError_t e = with_shape(bf16_io, s, BwdCall{x, xs, w, dy, dx, part, M, H, D, eps, p, st});
  if (e != hipSuccess) return e;
  return column_sum_launch(part, p.P, 2 * H * D, StoreNormGrads{dw, db, H * D}, st);
}

}  // namespace ttt
