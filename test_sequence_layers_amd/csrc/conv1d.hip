// Short causal depth-wise convolution over the tokens of [B, N, C], forward, backward and one token at a
// time: K = 2..4 taps per channel over the token and the K - 1 before it, then optionally SiLU.
//   pre[n] = bias + sum_k w[k] x[n - (K - 1) + k],   y = pre or pre sigmoid(pre)
//   dpre = dy act'(pre),  dx[n] = sum_k w[k] dpre[n + K - 1 - k],  dw[k] = sum dpre[n] x[n - (K - 1) + k]
//
// A stream bound by HBM. A thread owns four channels, 8 bytes of bf16 or 16 of fp32 (one channel where rows are not
// whole such pieces), and walks down a run of tokens with the last K inputs in registers, so that every
// input is read once but for the K - 1 tokens before each run (from L2). The next tokens are loaded while
// the last are worked on, and nothing in the walk branches: loads are clamped to the sequence and
// their values chosen, stores past the run write its last row again with the same value, so that no
// load is waited for together with a store behind it. The backward pass walks the same way with the last
// K values of dpre beside the inputs: dx lags K - 1 tokens behind. dw and db stay in registers over a run,
// are joined in LDS over the runs of a workgroup, and a second launch sums the workgroups' partial
// rows in a fixed order. bf16, K = 4, SiLU: forward of 2 x 16384 x 768 21.3 us (101 MB at 4.7 TB/s; a copy of as
// much takes 19.7), backward of 4 x 8192 x 768 36.2 us (151 MB at 4.2 TB/s; 29.6), 64 single tokens 3.3 us,
// which is the launch.
#include "internal.hpp"
#include "rowops.hpp"
#include "seq.hpp"

namespace ttt {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;     // tokens loaded ahead
constexpr int kPieces = 32;   // backward: pieces of a row per workgroup
constexpr int kRuns = kThreads / kPieces;  // backward: runs per workgroup

// Tokens per thread, a multiple of kAhead. Long runs read fewer tokens twice, short ones give more threads and
// end sooner: 1024 x 768 tokens and channels take 4.6 us forward (9.0 backward) in runs of 4, 5.6 (10.5) of 8
// and 11.0 (16.9) of 32; 8 x 1024 x 768 10.2 (20.6), 9.7 (18.2), 13.1 (19.5); 4 x 4096 x 768 13.9 (24.3) of 16,
// 14.2 (27.4) of 8, 16.0 (26.6) of 32; 4 x 8192 x 768 backward 36.5 of 32 and 39.4 of 16.
int run_length(int B, int N, int C) {
  const double all = (double)B * N * C;
  return all < (1 << 21) ? 4 : all < (1 << 23) ? 8 : all < (1 << 24) ? 16 : 32;
}

template <bool SILU>
__device__ __forceinline__ float act(float pre) {
  return SILU ? pre * sigmoid(pre) : pre;
}

// Input token t (t < n) of a sequence: the state's rows before token 0, zeros without a state.
template <class T, int V, int K>
__device__ __forceinline__ void input(const T* x, long long xs, const T* state, int C, int t, float* out) {
  if (t >= 0) {
    load_row<T, V>(x + (long long)t * xs, out);
  } else if (state) {
    load_row<T, V>(state + (long long)(K - 1 + t) * C, out);
  } else {
    for (int i = 0; i < V; ++i) out[i] = 0.f;
  }
}

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

template <int V, int K>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int c0, float (*wt)[V], float* bs) {
  for (int i = 0; i < V; ++i) {
    for (int k = 0; k < K; ++k) wt[k][i] = w[(long long)(c0 + i) * K + k];
    bs[i] = bias ? bias[c0 + i] : 0.f;
  }
}

template <class T, int V, int K, bool SILU>
__global__ __launch_bounds__(kThreads) void conv1d_fwd(Conv1dArgs a, int pieces, int runs, int len) {
  const long long id = ((long long)blockIdx.z * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (id >= (long long)pieces * runs) return;
  const int run = (int)(id / pieces), piece = (int)(id - (long long)run * pieces);
  const int b = blockIdx.y, C = a.C, c0 = piece * V;
  const int n = length_of(a.lengths, b, a.N);
  const T* x = (const T*)a.x + (long long)b * a.N * a.xs + c0;
  const T* state = a.state ? (const T*)a.state + (long long)b * (K - 1) * C + c0 : nullptr;
  T* y = (T*)a.y + (long long)b * a.N * C + c0;
  const int t0 = run * len, t1 = min(a.N, t0 + len);
  Raw<T, V> next[kAhead];
  auto fetch = [&](int t) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) next[j].load(x + (long long)max(min(t + j, n - 1), 0) * a.xs);
  };
  fetch(t0);
  float wt[K][V], bs[V], win[K][V], o[V];
  load_taps<V, K>(a.w, a.bias, c0, wt, bs);
  for (int k = 0; k < K - 1; ++k) input<T, V, K>(x, a.xs, state, C, min(t0, n) - (K - 1) + k, win[k]);
  if (run == 0 && a.state_out) {
    T* so = (T*)a.state_out + (long long)b * (K - 1) * C + c0;
    for (int j = 0; j < K - 1; ++j) {
      float v[V];
      input<T, V, K>(x, a.xs, state, C, n - (K - 1) + j, v);
      store_row<T, V>(so + (long long)j * C, v);
    }
  }
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int t = t0; t < t1; t += kAhead) {
    Raw<T, V> cur[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) cur[j] = next[j];
    fetch(t + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      cur[j].widen(win[K - 1]);
      const bool in = t + j < n, mine = t + j < t1;
      for (int i = 0; i < V; ++i) {
        float s = bs[i];
        for (int k = 0; k < K; ++k) s = fmaf(wt[k][i], win[k][i], s);
        o[i] = mine ? (in ? act<SILU>(s) : 0.f) : o[i];
        for (int k = 0; k < K - 1; ++k) win[k][i] = win[k + 1][i];
      }
      store_row<T, V>(y + (long long)min(t + j, t1 - 1) * C, o);
    }
  }
}

template <class T, int V, int K, bool SILU>
__global__ __launch_bounds__(kThreads) void conv1d_step(Conv1dArgs a, int pieces) {
  const long long id = wide_block() * kThreads + threadIdx.x;
  if (id >= (long long)pieces * a.B) return;
  const int b = (int)(id / pieces), c0 = (int)(id - (long long)b * pieces) * V, C = a.C;
  const T* st = (const T*)a.state + (long long)b * (K - 1) * C + c0;
  T* so = (T*)a.state_out + (long long)b * (K - 1) * C + c0;
  float wt[K][V], bs[V], win[K][V];
  for (int k = 0; k < K - 1; ++k) load_row<T, V>(st + (long long)k * C, win[k]);
  load_row<T, V>((const T*)a.x + (long long)b * a.xs + c0, win[K - 1]);
  load_taps<V, K>(a.w, a.bias, c0, wt, bs);
  float o[V];
  for (int i = 0; i < V; ++i) {
    float s = bs[i];
    for (int k = 0; k < K; ++k) s = fmaf(wt[k][i], win[k][i], s);
    o[i] = act<SILU>(s);
  }
  for (int k = 0; k < K - 1; ++k) store_row<T, V>(so + (long long)k * C, win[k + 1]);
  store_row<T, V>((T*)a.y + (long long)b * C + c0, o);
}

// Workgroup: kPieces pieces of the row x kRuns runs of one sequence. Partial row (b, run group):
// [K + 1][C], the K sums of dw and that of db.
template <class T, int V, int K, bool SILU>
__global__ __launch_bounds__(kThreads) void conv1d_bwd(Conv1dArgs a, int pieces, int len) {
  __shared__ float join[kRuns][kPieces * V];
  const int piece = blockIdx.y * kPieces + threadIdx.x % kPieces, sub = threadIdx.x / kPieces;
  const int b = blockIdx.z, C = a.C, c0 = piece * V;
  const bool live = piece < pieces;
  float acc[K + 1][V] = {};
  const long long first = ((long long)blockIdx.x * kRuns + sub) * len;
  if (live && first < a.N) {
    const int n = length_of(a.lengths, b, a.N);
    const T* x = (const T*)a.x + (long long)b * a.N * a.xs + c0;
    const T* state = a.state ? (const T*)a.state + (long long)b * (K - 1) * C + c0 : nullptr;
    const T* dy = (const T*)a.dy + (long long)b * a.N * C + c0;
    T* dx = (T*)a.dx + (long long)b * a.N * C + c0;
    const int t0 = (int)first, t1 = min(a.N, t0 + len), te = min(t1, n);
    Raw<T, V> nx[kAhead], nd[kAhead];
    auto fetch = [&](int t) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const long long tt = max(min(t + j, n - 1), 0);
        nx[j].load(x + tt * a.xs);
        nd[j].load(dy + tt * C);
      }
    };
    fetch(t0);
    float wt[K][V], bs[V], win[K][V], dp[K][V] = {}, o[V];
    load_taps<V, K>(a.w, a.bias, c0, wt, bs);
    for (int k = 0; k < K - 1; ++k) input<T, V, K>(x, a.xs, state, C, min(t0, n) - (K - 1) + k, win[k]);
    // One token: its dpre (none behind the sequence), its part of the parameters' gradients (of the run's
    // own tokens; not those behind the sequence, whose windows may hold a state or a last input that is not
    // finite), and o = dx[t - (K - 1)], which then has all it needs:
    // dp[k] = dpre[t - (K - 1) + k], dx[t - (K - 1)] = sum_k w[K - 1 - k] dp[k].
    auto token = [&](int t, const Raw<T, V>& rx, const Raw<T, V>& rd, float* out) {
      float d[V];
      rx.widen(win[K - 1]);
      rd.widen(d);
      const bool in = t < n;
      for (int i = 0; i < V; ++i) {
        win[K - 1][i] = in ? win[K - 1][i] : 0.f;
        if (SILU) {
          float pre = bs[i];
          for (int k = 0; k < K; ++k) pre = fmaf(wt[k][i], win[k][i], pre);
          const float s = sigmoid(pre);
          d[i] *= s * fmaf(pre, 1.f - s, 1.f);
        }
        d[i] = in ? d[i] : 0.f;
      }
      if (t < te)
        for (int i = 0; i < V; ++i) {
          acc[K][i] += d[i];
          for (int k = 0; k < K; ++k) acc[k][i] = fmaf(d[i], win[k][i], acc[k][i]);
        }
      for (int i = 0; i < V; ++i) {
        for (int k = 0; k < K - 1; ++k) win[k][i] = win[k + 1][i], dp[k][i] = dp[k + 1][i];
        dp[K - 1][i] = d[i];
        out[i] = 0.f;
        for (int k = 0; k < K; ++k) out[i] = fmaf(wt[K - 1 - k][i], dp[k][i], out[i]);
      }
    };
    // The first K - 1 tokens complete no dx of this run; a sequence's first run has the state's there.
    Raw<T, V> cx[kAhead], cd[kAhead];
    static_assert(K - 1 <= kAhead, "the tokens before the first dx are one fetch");
#pragma unroll
    for (int j = 0; j < kAhead; ++j) cx[j] = nx[j], cd[j] = nd[j];
    fetch(t0 + K - 1);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      token(t0 + j, cx[j], cd[j], o);
      if (t0 == 0 && a.dstate) store_row<T, V>((T*)a.dstate + ((long long)b * (K - 1) + j) * C + c0, o);
    }
    for (int t = t0; t < t1; t += kAhead) {  // t: the dx completed
#pragma unroll
      for (int j = 0; j < kAhead; ++j) cx[j] = nx[j], cd[j] = nd[j];
      fetch(t + K - 1 + kAhead);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        float v[V];
        token(t + K - 1 + j, cx[j], cd[j], v);
        for (int i = 0; i < V; ++i) o[i] = t + j < t1 ? v[i] : o[i];
        store_row<T, V>(dx + (long long)min(t + j, t1 - 1) * C, o);
      }
    }
  }
  float* row = a.partial + ((long long)b * gridDim.x + blockIdx.x) * (K + 1) * C;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
    for (int i = 0; i < V; ++i) join[sub][(threadIdx.x % kPieces) * V + i] = acc[k][i];
    __syncthreads();
    for (int t = threadIdx.x; t < kPieces * V; t += kThreads) {
      const int c = blockIdx.y * kPieces * V + t;
      if (c >= C) break;
      float s = 0.f;
      for (int q = 0; q < kRuns; ++q) s += join[q][t];
      row[(long long)k * C + c] = s;
    }
  }
}

template <int K>
struct StoreConvGrads {
  float *dw, *db;
  int C;
  __device__ void operator()(int col, float s) const {
    const int k = col / C, c = col - k * C;
    if (k < K) dw[(long long)c * K + k] = s;
    else if (db) db[c] = s;
  }
};

// Four channels at a time (8 bytes of bf16, 16 of fp32) where every row starts on such a piece.
bool vector_rows(bool bf, const Conv1dArgs& a) {
  uintptr_t at = 0;
  for (const void* p : {a.x, a.state, (const void*)a.y, (const void*)a.state_out, a.dy, (const void*)a.dx,
                        (const void*)a.dstate})
    at |= reinterpret_cast<uintptr_t>(p);
  return a.C % 4 == 0 && a.xs % 4 == 0 && at % (bf ? 8 : 16) == 0;
}

int run_groups(int B, int N, int C) {
  const int per = run_length(B, N, C) * kRuns;
  return (int)(((long long)N + per - 1) / per);
}

// Calls f.run<T, V, K, SILU>().
template <class F>
hipError_t with_variant(bool bf, bool vec, int K, bool silu, const F& f) {
#define TTT_CONV(T, v, k) \
  if (K == k) return silu ? f.template run<T, v, k, true>() : f.template run<T, v, k, false>();
  if (bf) {
    if (vec) { TTT_CONV(bf16, 4, 2) TTT_CONV(bf16, 4, 3) TTT_CONV(bf16, 4, 4) }
    else { TTT_CONV(bf16, 1, 2) TTT_CONV(bf16, 1, 3) TTT_CONV(bf16, 1, 4) }
  } else {
    if (vec) { TTT_CONV(float, 4, 2) TTT_CONV(float, 4, 3) TTT_CONV(float, 4, 4) }
    else { TTT_CONV(float, 1, 2) TTT_CONV(float, 1, 3) TTT_CONV(float, 1, 4) }
  }
#undef TTT_CONV
  return hipErrorInvalidValue;
}

struct FwdCall {
  const Conv1dArgs& a;
  hipStream_t st;
  template <class T, int V, int K, bool SILU>
  hipError_t run() const {
    const int pieces = a.C / V, len = run_length(a.B, a.N, a.C), runs = (a.N + len - 1) / len;
    const long long blocks = ((long long)pieces * runs + kThreads - 1) / kThreads;
    const dim3 g = wide_grid(blocks);
    hipLaunchKernelGGL((conv1d_fwd<T, V, K, SILU>), dim3(g.x, (unsigned)a.B, g.y), dim3(kThreads), 0, st, a, pieces,
                       runs, len);
    return hipGetLastError();
  }
};

struct StepCall {
  const Conv1dArgs& a;
  hipStream_t st;
  template <class T, int V, int K, bool SILU>
  hipError_t run() const {
    const int pieces = a.C / V;
    const long long blocks = ((long long)pieces * a.B + kThreads - 1) / kThreads;
    hipLaunchKernelGGL((conv1d_step<T, V, K, SILU>), wide_grid(blocks), dim3(kThreads), 0, st, a, pieces);
    return hipGetLastError();
  }
};

struct BwdCall {
  const Conv1dArgs& a;
  hipStream_t st;
  template <class T, int V, int K, bool SILU>
  hipError_t run() const {
    const int pieces = a.C / V, groups = run_groups(a.B, a.N, a.C);
    const dim3 grid((unsigned)groups, (unsigned)((pieces + kPieces - 1) / kPieces), (unsigned)a.B);
    hipLaunchKernelGGL((conv1d_bwd<T, V, K, SILU>), grid, dim3(kThreads), 0, st, a, pieces,
                       run_length(a.B, a.N, a.C));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return column_sum_launch(a.partial, (long long)a.B * groups, (K + 1) * a.C, StoreConvGrads<K>{a.dw, a.db, a.C}, st);
  }
};

}  // namespace

hipError_t conv1d_launch(bool bf16_io, int K, bool silu, const Conv1dArgs& a, hipStream_t st) {
  return with_variant(bf16_io, vector_rows(bf16_io, a), K, silu, FwdCall{a, st});
}

hipError_t conv1d_step_launch(bool bf16_io, int K, bool silu, const Conv1dArgs& a, hipStream_t st) {
  return with_variant(bf16_io, vector_rows(bf16_io, a), K, silu, StepCall{a, st});
}

size_t conv1d_bwd_workspace_bytes(bool, int B, int N, int C, int K) {
  return (size_t)B * run_groups(B, N, C) * (K + 1) * C * sizeof(float);
}

hipError_t conv1d_bwd_launch(bool bf16_io, int K, bool silu, const Conv1dArgs& a, hipStream_t st) {
  return with_variant(bf16_io, vector_rows(bf16_io, a), K, silu, BwdCall{a, st});
}

}  // namespace ttt
