// RMS norm over each head's D channels, forward and backward, with the residual's addition (and dropout of what is added)
// before it and, forward, an output in 8 bits after it.
//   s = residual + x keep / (1 - p),  y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   e4m3: q = y / scale,  scale = max |y| over a row or a group of its channels / 448
//   ds = dsum + rstd (g - xhat mean(g xhat)),  g = dy w,  xhat = s rstd;   dx = ds keep / (1 - p);   dw = sum dy xhat.
//
// A stream of rows, bound by HBM, laid out as layer norm's (normrows.hpp): a row is read once into the registers of L
// lanes, and the sum, the statistics, the maxima and every output come from there. Apart, the addition, the norm and
// the conversion would read and write the row two more times each. At the card's copying rate (5.2 TB/s) or near it: 32768 x 768 in bf16
// with dropout forward 36.7 us (5.5 TB/s), backward 52 (4.9); 16384 x 1536 into 8 bits 34 in groups of 128 and 33 by rows (5.2 and
// 5.3). Small calls are a launch: 16 x 768 into 8 bits 3.7 us, backward 1537 x 1001 in fp32 12.2 (one row a wave, then 3 us for the sum
// of partial rows).
#include "internal.hpp"
#include "lm.hpp"
#include "normrows.hpp"
#include "philox.hpp"
#include "pieces.hpp"

namespace ttt {
namespace {

// Where a row's D elements are over L lanes: piece k L + lane of access k. Where D is no multiple of V, the last piece, in access PART,
// is a part of one: its lane has the row's last V elements, in an access like the others, of which the first `skip` are the piece's
// before it and count as none here (where a row is less than a piece, there are none). PART is -1 where there is no such piece.
template <int L, int V, int PART>
struct Spread {
  static constexpr bool kTail = PART >= 0;
  int lane, D, whole, rest, skip;  // whole pieces; elements behind them
  __device__ __forceinline__ Spread(int lane, int D)
      : lane(lane), D(D), whole(D / V), rest(D % V), skip(kTail && lane == whole % L ? V - rest : 0) {}
  static constexpr __device__ bool has_part(int k) { return k == PART; }
  __device__ __forceinline__ bool full(int k) const { return kTail && k != PART ? k < PART : k * L + lane < whole; }
  __device__ __forceinline__ bool any(int k) const { return has_part(k) ? (k * L + lane) * V < D : full(k); }
  __device__ __forceinline__ bool part(int k) const { return has_part(k) && skip > 0; }
  __device__ __forceinline__ bool holds(int k, int i) const { return any(k) && (!has_part(k) || i >= skip); }
  // The channel of access k's first element; past the row its first.
  __device__ __forceinline__ int from(int k) const { return full(k) ? (k * L + lane) * V : any(k) ? D - V : 0; }
};

template <class T, int L, int K, int PART>
struct AnyRow {
  static constexpr int V = kPiece<T>;
  typedef Spread<L, V, PART> S;
  Piece<T> r[K];
  __device__ __forceinline__ void load(const T* p, const S& s) {
    if (PART == 0 && s.whole == 0) {
      if (s.lane == 0) r[0].load_last(p, s.rest);
      return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) r[k].load(p + s.from(k));
  }
  __device__ __forceinline__ void widen(float* v, const S& s, bool in = true) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      r[k].widen(v + k * V);
      for (int i = 0; i < V; ++i) v[k * V + i] = in && s.holds(k, i) ? v[k * V + i] : 0.f;
    }
  }
  static __device__ __forceinline__ void store(T* p, const float* v, const S& s) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (s.full(k)) Piece<T>::store(p + (k * L + s.lane) * V, v + k * V);
      if (s.part(k)) Piece<T>::store_last(p + s.whole * V, v + k * V, s.rest);
    }
  }
};

// The fp32 weights of a row's elements.
template <int L, int K, int V, int PART>
__device__ __forceinline__ void load_weights(const float* w, float* out, const Spread<L, V, PART>& s) {
  if (PART == 0 && s.whole == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = s.holds(0, i) ? w[s.from(0) + i] : 0.f;
    return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    for (int i = 0; i < V; i += 4) {
      Piece<float> q;
      q.load(w + s.from(k) + i);
      q.widen(out + k * V + i);
    }
}

// rstd of a row, over *back: v is multiplied by *back where its squares overflow (from 2^60 or so on: the largest squares are 2^96
// then, and eps is nothing beside them) or are next to nothing under an eps that is too (their sum and eps below 2^-90: the smallest numbers
// become 2^-41, the largest squares 2^126), so that such rows are normed like others. An infinite or NaN entry makes its row NaN at least
// where the entry is.
template <int L, int K, int V>
__device__ __forceinline__ float inverse_rms(float* v, int D, float eps, float (*red)[16], float* back) {
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < K * V; ++j) q = fmaf(v[j], v[j], q);
  q = row_sum<L>(q, red, 0);
  *back = 1.f;
  const bool over = !(q < __builtin_inff()), under = q < 0x1p-90f && eps < 0x1p-90f;
  if (__ballot(over || under)) {  // (rows of more than a wave: the same for all of it)
    const float by = over ? 0x1p-80f : under ? 0x1p108f : 1.f;
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < K * V; ++j) {
      v[j] *= by;
      t = fmaf(v[j], v[j], t);
    }
    q = row_sum<L>(t, red, 1);
    eps = over ? 0.f : eps * by * by;
    *back = by;
  }
  return rcp_hw(sqrtf(fmaf(q, rcp_hw((float)D), eps)));
}

// v -> v keep scale. (The mask costs 1.4 us of 36.7 forward at 32768 x 768.)
template <int L, int K, int V, int PART>
__device__ __forceinline__ void drop_row(float* v, const Drop& d, long long row, const Spread<L, V, PART>& s) {
  RowMask<L, K, V> m;
  m.make(d.rng[0], d.rng[1] + (unsigned long long)row * (unsigned)((s.D + 7) / 8), d.least, s.lane);
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (s.has_part(k)) m.bits[k] <<= s.skip;
#pragma unroll
  for (int k = 0; k < K; ++k)
    for (int i = 0; i < V; ++i) v[k * V + i] = m.kept(k, i) ? v[k * V + i] * d.scale : 0.f;
}

// Largest value over aligned groups of L lanes (runtime L, a power of two, 4 at least: 32 channels of bf16).
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int L) {
  auto other = [](uint32_t a, int which) {
    const int x = (int)a;
    return (uint32_t)(which == 1 ? __builtin_amdgcn_update_dpp(0, x, kDppXor1, 0xf, 0xf, true)
                      : which == 2 ? __builtin_amdgcn_update_dpp(0, x, kDppXor2, 0xf, 0xf, true)
                      : which == 4 ? __builtin_amdgcn_update_dpp(0, x, kDppMirror8, 0xf, 0xf, true)
                                   : __builtin_amdgcn_update_dpp(0, x, kDppMirror16, 0xf, 0xf, true));
  };
  v = max(v, other(v, 1));
  v = max(v, other(v, 2));
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
__device__ __forceinline__ uint32_t to_e4m3(const float* v) {
  const int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
}
// Halfway between two numbers of e4m3, from 2^-6 on, and of any size: 20 bits of fp32's fraction are past theirs, and below 2^-6, where
// their steps stay 2^-9, one more for each halving. (The second is for waves that have one of the first or a number below 2^-6: 16384 x 1536 in groups of
// 128 33.8 us, 33.3 with the first alone.)
__device__ __forceinline__ bool is_normal_tie(float v) { return (__float_as_uint(v) & 0xfffffu) == 0x80000u; }
__device__ __forceinline__ bool is_tie(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  const int past = 20 + max(0, 121 - (int)(u >> 23));  // (of 2^-6 the exponent is 121)
  return past <= 24 && (((u & 0x7fffffu) | 0x800000u) & ((1u << past) - 1)) == 1u << (past - 1);
}
// The neighbour of such a number on the side of `rest`, what it lacks to the value that it was rounded from (less than 2^-40 of it is
// none: products are known to 2^-46). Rounding to fp32 comes to a halfway point, but not past it, so that the value's own nearest is kept.
__device__ __forceinline__ float towards(float v, float rest) {
  const int u = __float_as_int(v), up = (__float_as_int(rest) ^ u) >= 0 ? 1 : -1;
  return __int_as_float(fabsf(rest) < 0x1p-40f * fabsf(v) ? u : u + up);
}
template <int K, int L, int V, int PART>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* v, const Spread<L, V, PART>& s) {
  typedef uint32_t Any __attribute__((aligned(1)));
  typedef uint16_t HalfWord __attribute__((aligned(1)));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    uint32_t q[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) q[i] = to_e4m3(v + k * V + 4 * i);
    if (s.full(k)) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) reinterpret_cast<Any*>(p + (k * L + s.lane) * V)[i] = q[i];
    }
    if (s.part(k)) {
      uint8_t* to = p + s.whole * V;
      uint64_t last = (V == 8 ? (uint64_t)q[V / 4 - 1] << 32 : 0) | q[0];
      last >>= 8 * s.skip;
      if (s.rest & 4) *reinterpret_cast<Any*>(to) = (uint32_t)last, to += 4, last >>= 32;
      if (s.rest & 2) *reinterpret_cast<HalfWord*>(to) = (uint16_t)last, to += 2, last >>= 16;
      if (s.rest & 1) *to = (uint8_t)last;
    }
  }
}

constexpr float kE4m3Most = 448.f;
constexpr float kLeastMax = 0x1p-100f;  // a smaller maximum's inverse could be infinite; such values are zeros in 8 bits

template <class T, int L, int K, int PART, bool ADD, bool E4M3>
__global__ __launch_bounds__(threads_of<L>) void rmsnorm_fwd(const T* __restrict__ x, long long xs, const T* res,
                                                             const float* __restrict__ w, T* sum, void* __restrict__ y,
                                                             float* __restrict__ scales, int rows, int H, int D,
                                                             int group, float eps, Drop drop) {
  constexpr int V = kPiece<T>;
  __shared__ float red[2][16];
  const Spread<L, V, PART> s(threadIdx.x % L, D);
  const long long row = wide_block() * (threads_of<L> / L) + threadIdx.x / L;
  if (row >= rows) return;  // (whole groups; for L > 64 the whole workgroup)
  const int m = (int)(row / H), h = (int)(row - (long long)m * H);
  AnyRow<T, L, K, PART> rx, rr;
  rx.load(x + (long long)m * xs + (long long)h * D, s);
  if (ADD) rr.load(res + row * D, s);
  float v[K * V], wv[K * V];
  rx.widen(v, s);
  if (ADD) {
    if (drop.least) drop_row<L, K>(v, drop, row, s);
    float r[K * V];
    rr.widen(r, s);
#pragma unroll
    for (int j = 0; j < K * V; ++j) v[j] += r[j];
    AnyRow<T, L, K, PART>::store(sum + row * D, v, s);
  }
  load_weights<L, K>(w + (long long)h * D, wv, s);
  float back;
  const float rstd = inverse_rms<L, K, V>(v, D, eps, red, &back);
  if constexpr (!E4M3) {
#pragma unroll
    for (int j = 0; j < K * V; ++j) v[j] *= rstd * wv[j];
    AnyRow<T, L, K, PART>::store((T*)y + row * D, v, s);
  } else {
    // rstd is not in y / scale: of v w, its maximum M over the group and 448 / M, the first and the last as two numbers
    // each, so that the rounding to 8 bits has but one other before it. v comes by the power of two 8 to 16 times below rstd, so that the
    // products are of the output's size and pass fp32 at neither end where that does not; `fine` is what is left of rstd (2^-66 stands below an
    // rstd of zero, of a row with an infinity). Maxima of the
    // absolute values' bits: as numbers they are in the same order, and a NaN is above all.
    const uint32_t part = max(__float_as_uint(rstd) & 0x7f800000u, 0x20000000u) - 0x01800000u;
    const float coarse = __uint_as_float(part), fine = rstd * __uint_as_float(0x7f000000u - part);
    float low[K * V];
    uint32_t most[K], all = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      most[k] = 0;
      for (int i = 0; i < V; ++i) {
        const int j = k * V + i;
        v[j] *= coarse;
        const float t = v[j] * wv[j];
        low[j] = fmaf(v[j], wv[j], -t);
        v[j] = s.holds(k, i) ? t : 0.f;
        most[k] = max(most[k], __float_as_uint(v[j]) & 0x7fffffffu);
      }
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
      const float top = __uint_as_float(group == D ? all : lanes_max(most[k], share));
      const float scaled = top * fine;  // the largest of the norm's output
      float scale = scaled * (1.f / kE4m3Most);  // (divided: the remainder is exact)
      scale = fmaf(fmaf(-scale, kE4m3Most, scaled), 1.f / kE4m3Most, scale);
      const float r = rcp_hw(top), inv = kE4m3Most * r, inv_low = fmaf(-inv, top, kE4m3Most) * r;
      // Zeros, next to nothing, infinities, NaN. (Lanes past the row are none of them: what they have is not stored.)
      const bool odd = s.any(k) && !(scaled >= kLeastMax && scaled < __builtin_inff());
      bool tie = odd;
      uint32_t least = ~0u;  // of the numbers other than zero, their bits twice (without the sign) less one
      float h[V];
      for (int i = 0; i < V; ++i) {
        h[i] = fmaf(v[k * V + i], inv, fmaf(v[k * V + i], inv_low, low[k * V + i] * inv));
        tie = tie || is_normal_tie(h[i]);
        least = min(least, (__float_as_uint(h[i]) << 1) - 1);
      }
      if (__ballot(tie || least < 0x79000000u - 1) != 0) {  // (2^-6; each lane by itself: a row's bits do not go by its neighbours)
        const float most = scaled < kLeastMax ? kLeastMax : scaled, plain = kE4m3Most / most;
        for (int i = 0; i < V; ++i) {
          const int j = k * V + i;
          const float rest = fmaf(v[j], inv, -h[i]) + fmaf(v[j], inv_low, low[j] * inv);
          if (is_tie(h[i])) h[i] = towards(h[i], rest);
          if (odd) h[i] = v[j] * fine * plain;
        }
        if (odd) scale = most / kE4m3Most;
      }
      for (int i = 0; i < V; ++i) v[k * V + i] = h[i];
      const int at = (k * L + s.lane) * V;
      if (at < D && (group == D ? at == 0 : (s.lane & (share - 1)) == 0)) scales[(row * D + at) / group] = scale;
    }
    store_e4m3<K>((uint8_t*)y + row * D, v, s);
  }
}

// Workgroup (bx, by): as in layer norm's backward pass, R tokens at a time of the HB heads from by HB on. Partial row bx: dw (H D).
template <class T, int L, int K, int PART, bool ADD>
__global__ __launch_bounds__(bwd_threads(L, K* kPiece<T>)) void rmsnorm_bwd(const T* __restrict__ sum, long long ss,
                                                                            const float* __restrict__ w,
                                                                            const T* __restrict__ dy, const T* dsum, T* ds,
                                                                            T* __restrict__ dx, float* __restrict__ part,
                                                                            int M, int H, int D, int HB, int R, float eps,
                                                                            Drop drop) {
  constexpr int V = kPiece<T>, LKV = L * K * V;
  constexpr bool kRoom = L <= 256;  // (as in layer norm's backward pass)
  __shared__ float red[4][16];
  __shared__ float join[L <= 64 ? bwd_threads(L, K * V) * K * V : 1];
  const int g = threadIdx.x / L;
  const Spread<L, V, PART> s(threadIdx.x % L, D);
  const int r = g / HB, hg = blockIdx.y * HB + g % HB, h = min(hg, H - 1);
  const bool live = r < R && hg < H;
  const float inv_d = rcp_hw((float)D);
  float wv[K * V], aw[K * V] = {};
  if (kRoom) load_weights<L, K>(w + (long long)h * D, wv, s);
  AnyRow<T, L, K, PART> rx, rd, rr;
  auto fetch = [&](long long m) {  // (past the last token: the last again)
    const long long t = m < M ? m : M - 1;
    rx.load(sum + t * ss + (long long)h * D, s);
    rd.load(dy + (t * H + h) * D, s);
    if (ADD) rr.load(dsum + (t * H + h) * D, s);
  };
  const long long step = (long long)gridDim.x * R;
  if (kRoom) fetch((long long)blockIdx.x * R + r);
  for (long long m0 = (long long)blockIdx.x * R; m0 < M; m0 += step) {
    const long long m = m0 + r;
    const bool in = live && m < M;
    float v[K * V], d[K * V], e[K * V];
    if (!kRoom) fetch(m);
    rx.widen(v, s);
    rd.widen(d, s, in);
    if (ADD) rr.widen(e, s, in);
    if (kRoom) fetch(m + step);
    float back;
    const float rstd = inverse_rms<L, K, V>(v, D, eps, red, &back);
    if (!kRoom) load_weights<L, K>(w + (long long)h * D, wv, s);
    float s2 = 0.f;
#pragma unroll
    for (int j = 0; j < K * V; ++j) {
      v[j] *= rstd;  // xhat
      aw[j] += in ? d[j] * v[j] : 0.f;
      d[j] *= wv[j];  // g
      s2 = fmaf(d[j], v[j], s2);
    }
    s2 = row_sum<L>(s2, red, 2) * inv_d;
    float outer = rstd * back;
    if (__ballot(!(outer < __builtin_inff()))) {  // (of a row below 2^-128 it is past fp32, not what comes of it)
      const float by = outer < __builtin_inff() ? 1.f : 0x1p40f;
#pragma unroll
      for (int j = 0; j < K * V; ++j) d[j] *= by;
      s2 *= by, outer = by == 1.f ? outer : rstd * (back * 0x1p-40f);
    }
#pragma unroll
    for (int j = 0; j < K * V; ++j) d[j] = outer * (d[j] - v[j] * s2) + (ADD ? e[j] : 0.f);
    const long long o = (m * H + h) * D;
    if (in) AnyRow<T, L, K, PART>::store(ds + o, d, s);
    if (dx) {
      if (drop.least) drop_row<L, K>(d, drop, m, s);
      if (in) AnyRow<T, L, K, PART>::store(dx + o, d, s);
    }
  }
  const long long W = (long long)H * D;
  float* row = part + (long long)blockIdx.x * W;
  if constexpr (L > 64) {  // one group: its registers are the workgroup's sums
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int i = 0; i < V; ++i) {
        if (s.holds(k, i)) row[(long long)h * D + s.from(k) + i] = aw[k * V + i];
      }
  } else {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int i = 0; i < V; ++i)
        if (s.holds(k, i)) join[g * LKV + s.from(k) + i] = aw[k * V + i];
    __syncthreads();
    for (int t = threadIdx.x; t < HB * D; t += blockDim.x) {
      const int hh = t / D, at = t - hh * D;
      if (blockIdx.y * HB + hh >= H) break;
      float total = 0.f;
      for (int q = 0; q < R; ++q) total += join[(q * HB + hh) * LKV + at];
      row[(long long)(blockIdx.y * HB + hh) * D + at] = total;
    }
  }
}

struct StoreWeightGrad {
  float* dw;
  __device__ void operator()(int col, float s) const { dw[col] = s; }
};

// Calls f with the access that has a part of a piece; of as many lanes' accesses as shape_of takes it is the last, of four one of two.
template <int L, int K, int V, class F>
hipError_t by_part(int D, const F& f) {
  if (D % V == 0) return f(std::integral_constant<int, -1>{});
  if constexpr (K == 4) {
    if (D / V / L == 2) return f(std::integral_constant<int, 2>{});
  }
  return D / V / L == K - 1 ? f(std::integral_constant<int, K - 1>{}) : hipErrorInvalidValue;
}

struct FwdCall {
  const RmsNormArgs& a;
  hipStream_t st;
  template <class T, int L, int K, int V>
  hipError_t run() const {
    return by_part<L, K, V>(a.D, [&](auto part) { return some<T, L, K, part.value>(); });
  }
  template <class T, int L, int K, int PART>
  hipError_t some() const {
    return a.scales ? (a.residual ? go<T, L, K, PART, true, true>() : go<T, L, K, PART, false, true>())
                    : (a.residual ? go<T, L, K, PART, true, false>() : go<T, L, K, PART, false, false>());
  }
  template <class T, int L, int K, int PART, bool ADD, bool E4M3>
  hipError_t go() const {
    constexpr int G = threads_of<L> / L;
    const int rows = a.M * a.H;
    hipLaunchKernelGGL((rmsnorm_fwd<T, L, K, PART, ADD, E4M3>), wide_grid(((long long)rows + G - 1) / G), dim3(threads_of<L>), 0,
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
    return by_part<L, K, V>(a.D, [&](auto part) {
      return a.dsum ? go<T, L, K, part.value, true>() : go<T, L, K, part.value, false>();
    });
  }
  template <class T, int L, int K, int PART, bool ADD>
  hipError_t go() const {
    const int threads = L <= 64 ? (p.HB * p.R * L + 63) / 64 * 64 : L;
    hipLaunchKernelGGL((rmsnorm_bwd<T, L, K, PART, ADD>), dim3((unsigned)p.P, (unsigned)p.gy), dim3(threads), 0, st,
                       (const T*)a.x, a.xs, a.w, (const T*)a.dy, (const T*)a.dsum, (T*)a.ds, (T*)a.dx, a.partial, a.M,
                       a.H, a.D, p.HB, p.R, a.eps, a.drop);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t rmsnorm_launch(bool bf16_io, const RmsNormArgs& a, hipStream_t st) {
  return with_pieces(bf16_io, shape_of(bf16_io, true, a.D), FwdCall{a, st});
}

size_t rmsnorm_bwd_workspace_bytes(bool bf16_io, int M, int H, int D) {
  return (size_t)bwd_plan(shape_of(bf16_io, true, D), M, H).P * H * D * sizeof(float);
}

hipError_t rmsnorm_bwd_launch(bool bf16_io, const RmsNormArgs& a, hipStream_t st) {
  const Shape s = shape_of(bf16_io, true, a.D);
  const BwdPlan p = bwd_plan(s, a.M, a.H);
  const hipError_t e = with_pieces(bf16_io, s, BwdCall{a, p, st});
  if (e != hipSuccess) return e;
  return column_sum_launch(a.partial, p.P, a.H * a.D, StoreWeightGrad{a.dw}, st);
}

}  // namespace ttt
