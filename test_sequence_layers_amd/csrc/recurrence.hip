// Gated linear recurrence: forward, one token at a time, and backward. Per channel,
//   la = -scale softplus(lam) sigmoid(r),  a = exp(la),  m = sqrt(1 - a^2),  h = a h + m sigmoid(i) x,  y = h.
// Backward, with q_n = dy_n + a_{n+1} q_{n+1}:
//   dx = q m sig(i),  di = q m x sig(i) (1 - sig(i)),  t = q (a la h_{n-1} - a^2 (la / m) sig(i) x),
//   dr = t (1 - sig(r)),  dlam = sum t sig(lam) / softplus(lam),  dh0 = a_0 q_0.
// t is la times the gradient of la: m's derivative -a^2 / m is infinite where a is 1, but la / m goes to 0 there
// with the root of la.
//
// A thread walks a channel of a sequence from end to end.
#include <type_traits>

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

// V neighbouring channels of one token as they are loaded (V = 2: 4 or 8 bytes), and stores of them.
template <class T, int V>
struct Pair {
  typedef typename std::conditional<sizeof(T) * V == 8, uint2, typename std::conditional<sizeof(T) * V == 4, uint32_t, uint16_t>::type>::type Bits;
  Bits b;
  __device__ __forceinline__ void load(const T* p) { b = *reinterpret_cast<const Bits*>(p); }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(Bits) == 8) return __uint_as_float(i ? b.y : b.x);
    else if constexpr (sizeof(T) == 4) return __uint_as_float(b);
    else return __uint_as_float(i ? (uint32_t)b & 0xffff0000u : (uint32_t)b << 16);
  }
  static __device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (V == 1) {
      p[0] = (T)v[0];
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
      typedef __bf16 two __attribute__((ext_vector_type(2)));
      typedef float ftwo __attribute__((ext_vector_type(2)));
      *reinterpret_cast<two*>(p) = __builtin_convertvector(ftwo{v[0], v[1]}, two);
    }
  }
};

// ---- what tiles tell each other ---------------------------------------------------------------
// A tile of a column (64 V channels of a sequence) tells the later ones its (decay, end) pairs, and every kGroup-th its
// end state: 64-bit words that are all ones until they are there, written and read whole by device-scope atomics, so that a word
// says by itself that it has come. A NaN is told as the one NaN that is not all ones.
constexpr int kGroup = 32;
constexpr unsigned long long kNotYet = ~0ull;
constexpr int kMostPolls = 1 << 22;

__device__ __forceinline__ uint32_t word_of(float v) { return v == v ? __float_as_uint(v) : 0x7fc00000u; }
__device__ __forceinline__ void tell(unsigned long long* p, float lo, float hi) {
  __hip_atomic_store(p, (unsigned long long)word_of(hi) << 32 | word_of(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long ask(const unsigned long long* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Words: a ticket counter, then [tiles][channels] pairs and [groups][channels] states of every sequence.
struct Board {
  unsigned* ticket;
  unsigned long long *pairs, *states;
};
__global__ void clear_board(unsigned long long* p, long long words) {
  for (long long k = (long long)blockIdx.x * blockDim.x + threadIdx.x; k < words; k += (long long)gridDim.x * blockDim.x)
    p[k] = k == 0 ? 0ull : kNotYet;
}

constexpr int kWaves = 8;  // of a workgroup
template <class T>
constexpr int kTokens = sizeof(T) == 2 ? 16 : 8;  // of a lane

template <class T, int V>
__global__ __launch_bounds__(64 * kWaves) void recurrence_fwd(RecurrenceArgs a, int tiles, int columns, Board board) {
  constexpr int TW = kTokens<T>, W = kWaves, TILE = TW * W, CH = 64 * V;
  __shared__ float2 part[W][CH], back[kGroup][CH];
  __shared__ float begin[CH];
  __shared__ unsigned drawn;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, C = a.C, N = a.N;
  // Tickets are drawn in the order in which workgroups start, and a tile waits for tiles of smaller tickets alone: they have
  // started and wait for still smaller ones, so that every wait ends.
  unsigned id = (unsigned)wide_block();
  if (tiles > 1) {
    if (threadIdx.x == 0) drawn = atomicAdd(board.ticket, 1u);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(drawn);
  }
  if (id >= (unsigned)(tiles * columns) * a.B) return;
  const int tile = id / (unsigned)(columns * a.B), rest = id - tile * (columns * a.B);
  const int b = rest / columns, column = rest - b * columns;
  const int c0 = column * CH + lane * V, c = min(c0, C - V);  // (past the last channel: the last ones again)
  const bool mine = c0 < C;
  const int n = length_of(a.lengths, b, N), t0 = tile * TILE + wave * TW;
  const long long row0 = (long long)b * N;
  T* y = (T*)a.y;
  float A[V], e[V];
  float av[TW][V], bv[TW][V];
  if (t0 < n) {
    Pair<T, V> x[TW], r[TW], g[TW];
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const long long at = row0 + min(t0 + t, N - 1);
      x[t].load((const T*)a.x + at * a.xs + c);
      r[t].load((const T*)a.r + at * a.rs + c);
      g[t].load((const T*)a.i + at * a.is + c);
    }
    float k[V];
    for (int i = 0; i < V; ++i) k[i] = a.scale * softplus(a.lam[c + i]), A[i] = 1.f, e[i] = 0.f;
#pragma unroll
    for (int t = 0; t < TW; ++t)
      for (int i = 0; i < V; ++i) {
        const Gates q(r[t].get(i), g[t].get(i), k[i]);
        const bool live = t0 + t < n;
        av[t][i] = live ? q.a : 1.f;
        bv[t][i] = live ? sqrtf(q.w) * q.gi * x[t].get(i) : 0.f;
        A[i] *= av[t][i];
        e[i] = fmaf(av[t][i], e[i], bv[t][i]);
      }
  } else {
    for (int i = 0; i < V; ++i) A[i] = 1.f, e[i] = 0.f;
  }
  const bool dead = tile * TILE >= n && tile > 0;  // nothing but padding
  if (!dead) {
    for (int i = 0; i < V; ++i) part[wave][lane * V + i] = make_float2(A[i], e[i]);
    __syncthreads();
    // The pair of the waves before this one; of the whole tile in the last.
    float pa[V], pe[V];
    for (int i = 0; i < V; ++i) pa[i] = 1.f, pe[i] = 0.f;
    for (int w = 0; w < wave; ++w)
      for (int i = 0; i < V; ++i) {
        const float2 p = part[w][lane * V + i];
        pa[i] *= p.x, pe[i] = fmaf(p.x, pe[i], p.y);
      }
    float ta[V], te[V];
    const long long word0 = ((long long)b * tiles) * (columns * CH) + column * CH + lane * V;
    if (wave == W - 1) {
      for (int i = 0; i < V; ++i) ta[i] = pa[i] * A[i], te[i] = fmaf(A[i], pe[i], e[i]);
      if (tile < tiles - 1)
        for (int i = 0; i < V; ++i) tell(board.pairs + word0 + (long long)tile * (columns * CH) + i, ta[i], te[i]);
    }
    const int first = tile / kGroup * kGroup, count = tile - first;
    for (int j = wave; j < count; j += W) {
      const unsigned long long* p = board.pairs + word0 + (long long)(first + j) * (columns * CH);
      unsigned long long v[V];
      for (int polls = 0; polls < kMostPolls; ++polls) {
        bool there = true;
        for (int i = 0; i < V; ++i) v[i] = ask(p + i), there = there && v[i] != kNotYet;
        if (__all(there)) break;
        __builtin_amdgcn_s_sleep(1);
      }
      for (int i = 0; i < V; ++i)
        back[j][lane * V + i] = make_float2(__uint_as_float((uint32_t)v[i]), __uint_as_float((uint32_t)(v[i] >> 32)));
    }
    if (count > 0) __syncthreads();
    if (wave == W - 1) {
      float h[V];
      const long long group0 = ((long long)b * ((tiles + kGroup - 1) / kGroup)) * (columns * CH) + column * CH + lane * V;
      if (first > 0) {
        const unsigned long long* p = board.states + group0 + (long long)(first / kGroup - 1) * (columns * CH);
        unsigned long long v[V];
        for (int polls = 0; polls < kMostPolls; ++polls) {
          bool there = true;
          for (int i = 0; i < V; ++i) v[i] = ask(p + i), there = there && v[i] != kNotYet;
          if (__all(there)) break;
          __builtin_amdgcn_s_sleep(1);
        }
        for (int i = 0; i < V; ++i) h[i] = __uint_as_float((uint32_t)v[i]);
      } else {
        for (int i = 0; i < V; ++i) h[i] = a.h0 ? a.h0[(long long)b * C + c + i] : 0.f;
      }
      for (int j = 0; j < count; ++j)
        for (int i = 0; i < V; ++i) {
          const float2 p = back[j][lane * V + i];
          h[i] = fmaf(p.x, h[i], p.y);
        }
      for (int i = 0; i < V; ++i) {
        begin[lane * V + i] = h[i];
        const float end = fmaf(ta[i], h[i], te[i]);
        if (tile % kGroup == kGroup - 1 && tile < tiles - 1)
          tell(board.states + group0 + (long long)(tile / kGroup) * (columns * CH) + i, end, 0.f);
        if (a.h_out && mine && (tile + 1) * TILE >= n) a.h_out[(long long)b * C + c + i] = end;
      }
    }
    __syncthreads();
    float h[V];
    for (int i = 0; i < V; ++i) h[i] = fmaf(pa[i], begin[lane * V + i], pe[i]);
    const int rows = (N + kKept - 1) / kKept;
    float* states = a.states ? a.states + (long long)b * rows * C + c : nullptr;
    if (states && mine && t0 % kKept == 0 && t0 < N)
      for (int i = 0; i < V; ++i) states[(long long)(t0 / kKept) * C + i] = h[i];
    if (t0 < n) {
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        float o[V];
        for (int i = 0; i < V; ++i) h[i] = fmaf(av[t][i], h[i], bv[t][i]), o[i] = t0 + t < n ? h[i] : 0.f;
        if (y && mine && t0 + t < N) Pair<T, V>::store(y + (row0 + t0 + t) * C + c, o);
      }
    } else if (y) {
      const float o[V] = {};
      for (int t = 0; t < TW; ++t)
        if (mine && t0 + t < N) Pair<T, V>::store(y + (row0 + t0 + t) * C + c, o);
    }
    // The states before padding's tokens in later tiles are the last.
    if (states && wave == W - 1 && mine && (tile + 1) * TILE >= n)
      for (int j = (tile + 1) * TILE / kKept; j < rows; ++j)
        for (int i = 0; i < V; ++i) states[(long long)j * C + i] = h[i];
  } else if (y) {
    const float o[V] = {};
    for (int t = 0; t < TW; ++t)
      if (mine && t0 + t < N) Pair<T, V>::store(y + (row0 + t0 + t) * C + c, o);
  }
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

// How a call is cut up: V channels a lane, tiles of a sequence, columns.
struct Plan {
  int V, tiles, columns;
};
template <class T>
Plan plan_of(int N, int C, bool pairs) {
  const int V = pairs ? 2 : 1, tile = kTokens<T> * kWaves;
  return {V, (N + tile - 1) / tile, (C + 64 * V - 1) / (64 * V)};
}
// Words of the board: the ticket's (16), then pairs and states.
long long board_words(const Plan& p, int B) {
  if (p.tiles == 1) return 0;
  const long long row = (long long)p.columns * 64 * p.V;
  return 16 + (long long)B * row * (p.tiles + (p.tiles + kGroup - 1) / kGroup);
}
template <class T>
size_t board_bytes(int B, int N, int C) {
  const long long one = board_words(plan_of<T>(N, C, false), B), two = board_words(plan_of<T>(N, C, true), B);
  return (size_t)(one > two ? one : two) * 8;
}

template <class T, int V>
hipError_t launch_fwd(const RecurrenceArgs& a, void* ws, hipStream_t st) {
  const Plan p = plan_of<T>(a.N, a.C, V == 2);
  const long long words = board_words(p, a.B), row = (long long)p.columns * 64 * V;
  unsigned long long* w = static_cast<unsigned long long*>(ws);
  const Board board{reinterpret_cast<unsigned*>(w), w + 16, w + 16 + a.B * row * p.tiles};
  if (p.tiles > 1) {
    const long long blocks = (words + 1023) / 1024;
    hipLaunchKernelGGL(clear_board, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, st, w, words);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((recurrence_fwd<T, V>), wide_grid((long long)p.tiles * p.columns * a.B), dim3(64 * kWaves), 0, st, a,
                     p.tiles, p.columns, board);
  return hipGetLastError();
}

// Two channels an access need rows of pairs.
template <class T>
bool paired(const RecurrenceArgs& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) | reinterpret_cast<uintptr_t>(a.i) |
                       reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dx) |
                       reinterpret_cast<uintptr_t>(a.dr) | reinterpret_cast<uintptr_t>(a.di);
  return ((a.C | a.xs | a.rs | a.is) & 1) == 0 && at % (2 * sizeof(T)) == 0;
}

}  // namespace

size_t recurrence_workspace_bytes(bool bf16_io, int B, int N, int C) {
  return bf16_io ? board_bytes<bf16>(B, N, C) : board_bytes<float>(B, N, C);
}

hipError_t recurrence_launch(bool bf16_io, const RecurrenceArgs& a, void* ws, hipStream_t st) {
  if (bf16_io) return paired<bf16>(a) ? launch_fwd<bf16, 2>(a, ws, st) : launch_fwd<bf16, 1>(a, ws, st);
  return paired<float>(a) ? launch_fwd<float, 2>(a, ws, st) : launch_fwd<float, 1>(a, ws, st);
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
