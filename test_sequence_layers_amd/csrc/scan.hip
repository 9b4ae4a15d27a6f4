// Selective state space scan: forward, one token at a time, and backward. Per channel c with S states,
//   dt = softplus(delta + dbias),  h[s] = exp(dt A[s]) h[s] + dt B[s] u,  y = (sum_s C[s] h[s] + D u) z sigmoid(z).
//
// The recurrence is linear in h, so a sequence is cut into segments: a first launch runs every segment
// from h = 0 and keeps its end state and its sum of dt (the segment's decay is exp(A sum dt)), a
// second folds the segments' (decay, end) pairs in order into each segment's start state, and a last
// one runs all segments again from their starts and writes y. A sequence of one segment needs the
// last only.
//
// A lane owns one channel with all its S states in registers, a wave 64 channels of one segment: B
// and C are then the same for the whole wave and come through scalar loads into SGPRs (B also as one element
// per lane, see outer()), the sum over the states stays inside the lane, and every access of u, delta, z and y is
// a contiguous run over channels. What bounds it is the vector ALU: one exponential (half rate) and four multiplies or
// multiply-adds per state and token, about 35 operations per token beside them, and the second run.
// 4 x 8192 x 768 x 16, bf16, gated: 179 us (traced one by one 74 the first run, 15 the fold, 100 the last, with
// the vector ALU and the matrix core busy 90 % of the time in both runs: 84 and 103 instructions a token and wave,
// where the recurrence and the sum over the states alone are 64 and 68), 201 MB at 1.1 TB/s; one run's operations
// alone take 77 us, the bytes 40. 3 x <= 1999 x 1000 x 32, fp32: 85 us (31, 17 and 37), of which 22 are the 129 MB of
// the segments' states.
//
// Tried and not kept: a scalar row of B and C held one token ahead behind a scheduling barrier (259 against
// 247 us); the waves of a workgroup on consecutive segments, joined through LDS so that the fold goes over
// groups of four (fold 15 -> 5.5 us, but the last run starts later by as much; wide states lose waves
// to the registers it takes: 2 x 4096 x 768 x 32 119 -> 128 us); the backward pass's products with B and C as
// outer products on the matrix core (7 to 17 % fewer instructions, the same times within 1 %); the sum over the
// states there (a matrix instruction per state, since a lane holds its channel's states: slower).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "internal.hpp"
#include "rowops.hpp"
#include "seq.hpp"

namespace ttt {
namespace {

constexpr int kWaves = 4;   // units per workgroup (forward)
constexpr int kTokens = 2;  // tokens loaded ahead (4: 3 % slower, 1: 5 %; with 8 states 3 % faster at 2 x 4096 x 768,
                            // 6 % slower at 2 x 333 x 193)
constexpr float kLn2 = 0.693147180559945309417f;

// log(1 + exp(x)) with e = exp(-|x|): max(x, 0) + log1p(e), and log1p(e) = 2 atanh(s) with s = e / (2 + e) <= 1/3,
// = s P(s^2). P interpolates 2 atanh(sqrt q) / sqrt q at the five Chebyshev points of [0, 1/9] (off by at most
// 4.1e-9 of it; with fp32's roundings log1p is within 2e-7), so that small e keeps its relative
// precision. e is returned for the derivative.
constexpr float kLog1pP[5] = {2.0f, 0.6666632294654846f, 0.4002459645271301f, 0.27965158224105835f, 0.28157779574394226f};
__device__ __forceinline__ float softplus_of(float x, float& e) {
  e = exp2_hw(-kLog2e * fabsf(x));
  const float s = e * rcp_hw(2.f + e), q = s * s;
  float p = kLog1pP[4];
  for (int i = 3; i >= 0; --i) p = fmaf(p, q, kLog1pP[i]);
  return fmaf(s, p, fmaxf(x, 0.f));
}
// The step; below with its derivative by delta.
__device__ __forceinline__ float step_of(float raw, int softplus) {
  float e;
  const float dt = softplus_of(raw, e);  // (chosen, not branched to: a branch would part the tokens of a chunk)
  return softplus ? dt : raw;
}
__device__ __forceinline__ float step_grad_of(float raw, int softplus, float& grad) {
  float e;
  const float dt = softplus_of(raw, e);
  grad = softplus ? (raw >= 0.f ? 1.f : e) * rcp_hw(1.f + e) : 1.f;
  return softplus ? dt : raw;
}

// A row piece of B or of C that is the same for the whole wave, as raw dwords by scalar loads: those of a chunk's
// tokens are asked for together, before the chunk's steps are computed, as far as SGPRs hold them
// (4 x 8192 x 768 x 16, bf16: 196 us, against 211 with each token's asked for where it is used).
typedef const __attribute__((address_space(4))) uint32_t* ScalarPtr;
template <class T, int SB>
struct Piece {
  static constexpr int W = SB * (int)sizeof(T) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* p) {
    const ScalarPtr q = (ScalarPtr)(uintptr_t)p;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = q[i];
  }
};
template <class T, int SB>
__device__ __forceinline__ void widen(const uint32_t* w, float* out) {
#pragma unroll
  for (int i = 0; i < SB; ++i) {
    if constexpr (sizeof(T) == 4) out[i] = __uint_as_float(w[i]);
    else out[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
}

// acc[s] += row[s] * x over 4 NB states, a lane's channel having its own x: the outer product of a row of B
// (state s in the lanes s of 64, from 4 AT on) and the wave's channels. Four states by one v_mfma_f32_4x4x1 of 16
// blocks: a block is four lanes, its rows four states, its columns the lanes' channels, and all blocks take the
// rows of the one that AT names. The products are fused and rounded once, as fmaf's are.
template <int AT, int NB>
__device__ __forceinline__ void outer(float row, float x, f32x4* acc) {
  acc[0] = __builtin_amdgcn_mfma_f32_4x4x1f32(row, x, acc[0], 4, AT, 0);
  if constexpr (NB > 1) outer<AT + 1, NB - 1>(row, x, acc + 1);
}

// Where B comes as one element per lane and through outer(), instead of as scalars. An outer product takes as long as its
// four multiplications (16 cycles), so it gains only where a token's scalars are more than the SGPRs hold ahead of
// their use: in the last run, which has C's as well, always; in the first from rows of 64 bytes on.
//                                              scalars   outer()
//   last run   2 x 4096 x 768 x 8, bf16           52 us      48 us
//              2 x 4096 x 768 x 16, bf16          69         66
//              3 x 1999 x 1000 x 32, fp32         52         36    (the run alone)
//              1 x 32768 x 1536 x 16, bf16       320        327    (the other way, by 2 %)
//   first run  2 x 2048 x 768 x 64, bf16         121        107
//              4 x 8192 x 768 x 32, bf16         307        303
//              4 x 8192 x 768 x 16, bf16          75         79    (the run alone; 32 bytes: scalars)
template <class T, int S, bool FINAL>
constexpr bool outer_rows = FINAL || S * sizeof(T) >= 64;

// Channel c of a row that is the same for the whole wave: the row's address in SGPRs, the lane's part of it
// in one 32-bit register. (The empty asm keeps the two apart: added up ahead of the loop they would be a
// 64-bit address per lane and tensor, advanced by vector additions.)
__device__ __forceinline__ uint32_t lane_part(int c, int size) {
  uint32_t off = (uint32_t)c * (uint32_t)size;
  asm volatile("" : "+v"(off));
  return off;
}
template <class T>
__device__ __forceinline__ float at(const T* row, uint32_t off) {
  return (float)*reinterpret_cast<const T*>(reinterpret_cast<const char*>(row) + off);
}
template <class T>
__device__ __forceinline__ void put(T* row, uint32_t off, float v) {
  *reinterpret_cast<T*>(reinterpret_cast<char*>(row) + off) = (T)v;
}

// A row pointer that walks down the tokens (by 64-bit additions; the row of a token would take a 64-bit
// product). It stays where it is when `on` is false.
template <class T>
struct Walk {
  const char* p;
  long long step;
  __device__ __forceinline__ Walk(const void* base, long long stride, long long row, int col)
      : p(reinterpret_cast<const char*>((const T*)base + row * stride + col)), step(stride * (long long)sizeof(T)) {}
  __device__ __forceinline__ const T* row() const { return reinterpret_cast<const T*>(p); }
  __device__ __forceinline__ void next(bool on = true) { p += on ? step : 0; }
};

constexpr long long kSimds = 1024;  // of 256 CUs
// No segment is longer where there is more than one, and none of the backward pass: its sums over tokens (the steps',
// and those of d_A, d_D and d_delta_bias) take one after the other in fp32, and further ones would drift. (32768 steps
// of 0.003: off by 5900 times 2^-24. A segment's 16 states, written and read three times, are 2 % of its rows' bytes.)
constexpr int kLongest = 2048;
constexpr long long kMostUnits = 1 << 22;
// How a call is cut up. Channel blocks: 64 channels of one group each.
struct Plan {
  int cbg, cb;      // channel blocks per group, in all
  int nseg, T;      // segments per sequence, tokens each
};

struct Unit {
  int b, seg, cb, g, c;  // c: this lane's channel (a block's lanes past its group repeat the first)
  bool live;
};
__device__ __forceinline__ Unit unit_of(int id, const Plan& p, int C, int G) {
  Unit u;
  u.cb = id % p.cb;
  const int rest = id / p.cb;
  u.seg = rest % p.nseg;
  u.b = rest / p.nseg;
  u.g = u.cb / p.cbg;
  const int cg = C / G, first = (u.cb - u.g * p.cbg) * 64;
  u.live = first + lane_id() < cg;
  u.c = u.g * cg + first + (u.live ? lane_id() : 0);
  return u;
}

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

// Forward. FINAL: from the segment's start state (ends, once folded; h0 or zeros for a single
// segment), writing y and h_out. Otherwise from zero, writing the end state and the sum of dt.
// ends: [B][nseg][S][C], sums: [B][nseg][C].
template <class T, int S, bool FINAL>
__global__ __launch_bounds__(64 * kWaves) void scan_fwd(ScanArgs a, Plan p, int units, float* __restrict__ ends,
                                                        float* __restrict__ sums) {
  // (64 states leave no registers for more: 107 us, 113 with two. Nor do two of C's rows of 128 bytes leave SGPRs:
  // 4 x 8192 x 768 x 32, fp32, 297 us, 306 with two in the last run as well.)
  constexpr int kTok = S <= 32 && (!FINAL || S * sizeof(T) <= 64) ? kTokens : 1;
  constexpr bool kOuter = outer_rows<T, S, FINAL>;
  const int id = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= units) return;
  const Unit un = unit_of(id, p, a.C, a.G);
  const int C = a.C, N = a.N, c = un.c;
  const int n = length_of(a.lengths, un.b, N);
  const int t0 = un.seg * p.T, t1 = min(N, t0 + p.T), te = min(t1, n);
  const long long row0 = (long long)un.b * N;
  T* y = (T*)a.y + row0 * C;
  const long long seg_at = ((long long)un.b * p.nseg + un.seg) * C;

  float A2[S];
  f32x4 h[S / 4];
  for (int s = 0; s < S; ++s) A2[s] = a.A[(long long)c * S + s] * kLog2e;
  if (FINAL && p.nseg > 1) {
    for (int s = 0; s < S; ++s) h[s / 4][s % 4] = ends[seg_at * S + (long long)s * C + c];
  } else if (FINAL && a.h0) {
    for (int s = 0; s < S; ++s) h[s / 4][s % 4] = a.h0[((long long)un.b * C + c) * S + s];
  } else {
    for (int s = 0; s < S; ++s) h[s / 4][s % 4] = 0.f;
  }
  const float db = a.dbias ? a.dbias[c] : 0.f, D = FINAL && a.D ? a.D[c] : 0.f;
  float sum = 0.f;
  // The next kTok tokens' rows are loaded before this kTok are worked on (past the end: the last row
  // again), without a branch: behind one the loads would be waited for where it ends. Without a gate
  // u's row stands in for z's.
  const bool gate = FINAL && a.z;
  Walk<T> wu(a.u, a.us, row0 + t0, 0), wd(a.delta, a.ds, row0 + t0, 0);
  Walk<T> wz(gate ? a.z : a.u, gate ? a.zs : a.us, row0 + t0, 0);
  Walk<T> wb(a.bm, a.bs, row0 + t0, un.g * S), wc(a.cm, a.cs, row0 + t0, un.g * S);
  T* py = y + (long long)t0 * C;
  float nu[kTok], nd[kTok], nz[kTok], nb[kTok];  // nb: state l % S of the token's B in lane l, when kOuter
  int tf = t0;  // the token fetched next
  auto fetch = [&](uint32_t off) {
    uint32_t off_b = 0;
    if constexpr (kOuter) off_b = lane_part(lane_id() % S, sizeof(T));
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      nu[j] = at(wu.row(), off);
      nd[j] = at(wd.row(), off);
      if (kOuter) nb[j] = at(wb.row(), off_b);
      if (FINAL) nz[j] = at(wz.row(), off);
      const bool more = ++tf < te;
      wu.next(more), wd.next(more);
      if (kOuter) wb.next(more);
      if (FINAL) wz.next(more);
    }
  };
  // kTok tokens from t on (all there when FULL). Lanes past their group repeat its block's first channel
  // in everything, stores too, so that the stores need no branch either: a load behind a store that may
  // or may not be there is waited for together with it.
  auto chunk = [&](int t, auto full) {
    constexpr bool FULL = decltype(full)::value;
    const uint32_t off = lane_part(c, sizeof(T));
    float cu[kTok], dt[kTok], cz[kTok], cb[kTok], out[kTok];
    Piece<T, S> pb[kTok], pc[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const bool more = FULL || t + j < te - 1;
      if constexpr (!kOuter) pb[j].load(wb.row()), wb.next(more);
      if constexpr (FINAL) pc[j].load(wc.row()), wc.next(more);
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      cu[j] = nu[j];
      if (kOuter) cb[j] = nb[j];
      if (FINAL) cz[j] = nz[j];
      dt[j] = step_of(nd[j] + db, a.softplus);
    }
    fetch(off);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (FULL || t + j < te) {
        const float dtu = dt[j] * cu[j];
        float mat[S];
        if constexpr (kOuter) {
#pragma unroll
          for (int s = 0; s < S; ++s) h[s / 4][s % 4] *= exp2_hw(dt[j] * A2[s]);
          outer<0, S / 4>(cb[j], dtu, h);
        } else {
          widen<T, S>(pb[j].w, mat);
#pragma unroll
          for (int s = 0; s < S; ++s) {
            h[s / 4][s % 4] = fmaf(exp2_hw(dt[j] * A2[s]), h[s / 4][s % 4], dtu * mat[s]);
          }
        }
        if constexpr (FINAL) {
          float o[2] = {};
          widen<T, S>(pc[j].w, mat);
#pragma unroll
          for (int s = 0; s < S; ++s) o[s & 1] = fmaf(mat[s], h[s / 4][s % 4], o[s & 1]);
          out[j] = o[0] + o[1];
        }
        if (!FINAL) sum += dt[j];
        // (64 states: 106 us with a token's work kept together, 115 mixed with the next one's)
        if (kOuter) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (FINAL) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        float o = fmaf(D, cu[j], out[j]);
        o = gate ? o * (cz[j] * sigmoid(cz[j])) : o;
        if (FULL || t + j < te) put(py, off, o);
        py += C;
      }
    }
  };
  if (t0 < te) fetch(lane_part(c, sizeof(T)));
  int t = t0;
  for (; t + kTok <= te; t += kTok) chunk(t, std::true_type{});
  if (t < te) chunk(t, std::false_type{});
  if (FINAL) {
    for (int t = max(t0, te); t < t1; ++t) put(y + (long long)t * C, lane_part(c, sizeof(T)), 0.f);
    if (a.h_out && un.seg == p.nseg - 1)
      for (int s = 0; s < S; ++s) a.h_out[((long long)un.b * C + c) * S + s] = h[s / 4][s % 4];
  } else {
    for (int s = 0; s < S; ++s) ends[seg_at * S + (long long)s * C + c] = h[s / 4][s % 4];
    sums[seg_at + c] = sum;
  }
}

// Folds the segments in order: ends[seg] becomes the segment's start state. One thread per (b, s, c).
// For the backward pass back (same layout) holds the segments' own contributions to a_0 q_0 of their
// first token, and becomes what flows into each segment from behind it; dh0 receives the first's.
constexpr int kFoldThreads = 64;  // (single waves: they spread over all CUs)
__global__ __launch_bounds__(kFoldThreads) void scan_fold(const float* __restrict__ A, const float* __restrict__ h0,
                                                          float* __restrict__ ends, float* __restrict__ back,
                                                          const float* __restrict__ sums, float* __restrict__ dh0,
                                                          int C, int S, int nseg) {
  const int id = blockIdx.x * kFoldThreads + threadIdx.x;
  if (id >= C * S) return;
  const int s = id / C, c = id - s * C, b = blockIdx.y;
  const float A2 = A[(long long)c * S + s] * kLog2e;
  const long long hat = ((long long)b * C + c) * S + s, step = (long long)S * C;
  const bool rev = blockIdx.z != 0;
  float* f = (rev ? back : ends) + (long long)b * nseg * step + id;
  const float* dts = sums + (long long)b * nseg * C + c;
  float x = !rev && h0 ? h0[hat] : 0.f;
  // kFold segments' pairs are loaded while the chain goes through the kFold before them.
  constexpr int kFold = 32;
  float own[kFold], dec[kFold];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kFold; ++i) {
      const int k = min(i0 + i, nseg - 1);
      const long long seg = rev ? nseg - 1 - k : k;
      own[i] = f[seg * step];
      dec[i] = dts[seg * C];
    }
  };
  fetch(0);
  for (int i0 = 0; i0 < nseg; i0 += kFold) {
    float o[kFold], d[kFold];
#pragma unroll
    for (int i = 0; i < kFold; ++i) o[i] = own[i], d[i] = exp2_hw(A2 * dec[i]);
    if (i0 + kFold < nseg) fetch(i0 + kFold);
    auto chain = [&](auto zero) {
      int left = nseg - i0;
      // (Its own in either chain: conditions shared by the two would take 64 SGPRs.)
      asm volatile("" : "+s"(left));
#pragma unroll
      for (int i = 0; i < kFold; ++i)
        if (i < left) {
          f[(rev ? nseg - 1 - i0 - i : i0 + i) * step] = x;
          x = decltype(zero)::value && x == 0.f ? o[i] : fmaf(d[i], x, o[i]);
        }
    };
    // Where steps times A are positive a decay may be infinite, and NaN with a state of zero, which has no part of it:
    // then these segments again, zeros kept out. (Chosen at every segment the choice is a third of the chain.)
    const float start = x;
    chain(std::false_type{});
    if (x != x) x = start, chain(std::true_type{});
  }
  if (rev && dh0) dh0[hat] = x;
}

// One token: S / 4 lanes per channel, four states each (one 16-byte access of the state). Bound by its
// traffic where it is large, by the launch where it is small: 64 x 1536 x 16 5.3 us (12.6 MB of states).
template <class T, int S, bool VEC>
__global__ __launch_bounds__(256) void scan_step(ScanArgs a) {
  constexpr int L = S / 4;
  const long long id = wide_block() * 256 + threadIdx.x;
  const long long row = id / L;  // b * C + c
  if (row >= (long long)a.B * a.C) return;  // (whole groups of L lanes)
  const int q = (int)(id % L), b = (int)(row / a.C), c = (int)(row - (long long)b * a.C);
  const int g = c / (a.C / a.G);
  float h[4], A[4], bv[4], cv[4];
  if (VEC) {
    load_params<4>(a.h0 + row * S + 4 * q, h);
    load_params<4>(a.A + (long long)c * S + 4 * q, A);
  } else {
    for (int i = 0; i < 4; ++i) h[i] = a.h0[row * S + 4 * q + i];
    for (int i = 0; i < 4; ++i) A[i] = a.A[(long long)c * S + 4 * q + i];
  }
  const T* bm = (const T*)a.bm + b * a.bs + (long long)g * S + 4 * q;
  const T* cm = (const T*)a.cm + b * a.cs + (long long)g * S + 4 * q;
  for (int i = 0; i < 4; ++i) bv[i] = (float)bm[i];
  for (int i = 0; i < 4; ++i) cv[i] = (float)cm[i];
  const float u = (float)((const T*)a.u)[b * a.us + c];
  const float z = a.z ? (float)((const T*)a.z)[b * a.zs + c] : 0.f;
  const float raw = (float)((const T*)a.delta)[b * a.ds + c] + (a.dbias ? a.dbias[c] : 0.f);
  const float dt = step_of(raw, a.softplus), dtu = dt * u;
  float y = 0.f;
  for (int i = 0; i < 4; ++i) {
    h[i] = fmaf(exp2_hw(dt * (A[i] * kLog2e)), h[i], dtu * bv[i]);
    y = fmaf(cv[i], h[i], y);
  }
  y = lanes_sum<L>(y);
  if (a.D) y = fmaf(a.D[c], u, y);
  if (a.z) y *= z * sigmoid(z);
  if (VEC) {
    *reinterpret_cast<float4*>(a.h_out + row * S + 4 * q) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
    for (int i = 0; i < 4; ++i) a.h_out[row * S + 4 * q + i] = h[i];
  }
  if (q == 0) ((T*)a.y)[row] = (T)y;
}

// ---- backward ---------------------------------------------------------------------------------
//   v = dy z sigmoid(z),  q_n = v_n C_n + a_{n+1} q_{n+1}  (from the last token back)
// scan_bwd_ends runs every segment once from h = 0, keeping the local state and the sum of dt at every
// kSub-th token (the checkpoints), the end state, and the segment's contribution to a_0 q_0 of its
// first token, sum_n (a_0 ... a_n) v_n C_n, whose running product shares the exponentials. scan_fold
// joins the segments in both directions. scan_bwd then takes the sub-chunks of a segment from its
// last to its first: it forms the sub-chunk's a and h in registers from the checkpoint (one more
// exponential per state and token) and walks back through them. 2 x 4096 x 768 x 16, bf16, gated: 147 us (traced
// one by one 38 the ends, 15 the fold, 92 the walk at three waves per SIMD, 9 the last sums), the vector ALU
// busy 82 % of the walk and 65 % of the ends; one exponential less and no checkpoints would be 58 us of
// operations, the bytes 17.

// Tokens per sub-chunk, states per wave and waves of a scan_bwd workgroup: kSub * SW values of each of a
// and h stay in a lane's registers. Eight states a wave share what a token costs a wave, but leave two waves per
// SIMD, where four leave three (2 x 4096 x 768, bf16, four and eight: 16 states 154 and 197 us, 32 279 and 250).
template <int S>
struct Bwd {
  static constexpr int SW = S >= 32 ? 8 : 4;
  static constexpr int NW = S / SW;
  static constexpr int kSub = 8;
};
constexpr int kBwdSub = 8;

// Buffers in the workspace.
struct BwdBufs {
  float* ends;   // [B][nseg][S][C]
  float* back;   // [B][nseg][S][C]
  float* sums;   // [B][nseg][C]
  float* ck;     // [B][nsub][S][C] local states at the sub-chunks' starts
  float* cksum;  // [B][nsub][C] sums of dt from the segment's start to the sub-chunk's
  float* mats;   // [B][N][CB][2 S] a channel block's sums for dB and dC
  float* part;   // [B][nseg][S C + 2 C] a segment's dA ([S][C]), dD, ddbias
  int nsub;      // sub-chunks per sequence
};

template <class T, int S, int SB>
__global__ __launch_bounds__(64 * kWaves) void scan_bwd_ends(ScanArgs a, Plan p, int units, BwdBufs w) {
  constexpr int kSub = Bwd<S>::kSub, kTok = kTokens;
  int id = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= units) return;
  constexpr int NB = S / SB;  // state blocks, one per wave
  const int s0 = id % NB * SB;
  const Unit un = unit_of(id / NB, p, a.C, a.G);
  const int C = a.C, N = a.N, c = un.c;
  const int n = length_of(a.lengths, un.b, N);
  const int t0 = un.seg * p.T, t1 = min(N, t0 + p.T), te = min(t1, n);
  const long long row0 = (long long)un.b * N;
  const bool gate = a.z;
  Walk<T> wu(a.u, a.us, row0 + t0, 0), wd(a.delta, a.ds, row0 + t0, 0), wv(a.dy, C, row0 + t0, 0);
  Walk<T> wz(gate ? a.z : a.u, gate ? a.zs : a.us, row0 + t0, 0);
  Walk<T> wb(a.bm, a.bs, row0 + t0, un.g * S + s0), wc(a.cm, a.cs, row0 + t0, un.g * S + s0);
  float A2[SB], h[SB], P[SB], q[SB];
  for (int s = 0; s < SB; ++s) {
    A2[s] = a.A[(long long)c * S + s0 + s] * kLog2e;
    h[s] = q[s] = 0.f;
    P[s] = 1.f;
  }
  const float db = a.dbias ? a.dbias[c] : 0.f;
  float sum = 0.f;
  auto checkpoint = [&](int t) {
    const long long k = (long long)un.b * w.nsub + t / kSub;
    for (int s = 0; s < SB; ++s) w.ck[(k * S + s0 + s) * C + c] = h[s];
    if (s0 == 0) w.cksum[k * C + c] = sum;
  };
  float nu[kTok], nd[kTok], nv[kTok], nz[kTok];
  int tf = t0;
  auto fetch = [&]() {
    const uint32_t off = lane_part(c, sizeof(T));
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      nu[j] = at(wu.row(), off);
      nd[j] = at(wd.row(), off);
      nv[j] = at(wv.row(), off);
      nz[j] = at(wz.row(), off);
      const bool more = ++tf < te;
      wu.next(more), wd.next(more), wv.next(more), wz.next(more);
    }
  };
  auto chunk = [&](int t, auto full) {
    constexpr bool FULL = decltype(full)::value;
    float dtu[kTok], dt[kTok], v[kTok];
    Piece<T, SB> pb[kTok], pc[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      pb[j].load(wb.row());
      pc[j].load(wc.row());
      const bool more = FULL || t + j < te - 1;
      wb.next(more), wc.next(more);
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      dt[j] = step_of(nd[j] + db, a.softplus);
      dtu[j] = dt[j] * nu[j];
      v[j] = gate ? nv[j] * (nz[j] * sigmoid(nz[j])) : nv[j];
    }
    // (the checkpoint's stores before the next loads: what is waited for next has them behind it anyway)
    if ((t - t0) % kSub == 0) checkpoint(t);
    fetch();
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (FULL || t + j < te) {
        float bv[SB], cv[SB];
        widen<T, SB>(pb[j].w, bv);
        widen<T, SB>(pc[j].w, cv);
#pragma unroll
        for (int s = 0; s < SB; ++s) {
          const float e = exp2_hw(dt[j] * A2[s]);
          h[s] = fmaf(e, h[s], dtu[j] * bv[s]);
          P[s] *= e;
          q[s] = fmaf(P[s], v[j] * cv[s], q[s]);
        }
        sum += dt[j];
      }
    }
  };
  if (t0 < te) fetch();
  int t = t0;
  for (; t + kTok <= te; t += kTok) chunk(t, std::true_type{});
  if (t < te) chunk(t, std::false_type{});
  // (the sub-chunks behind the sequence start from its end)
  for (t = t0 + (max(te - t0, 0) + kSub - 1) / kSub * kSub; t < t1; t += kSub) checkpoint(t);
  const long long seg = (long long)un.b * p.nseg + un.seg;
  for (int s = 0; s < SB; ++s) {
    w.ends[(seg * S + s0 + s) * C + c] = h[s];
    w.back[(seg * S + s0 + s) * C + c] = q[s];
  }
  if (s0 == 0) w.sums[seg * C + c] = sum;
}

// Sums over the 64 lanes, halving the values and the lanes that hold a part of each at every step: joined
// over lane bit M, lanes with that bit clear go on with x and the others with y. Bits 5 and 4 by swaps
// of register halves, the rest within 16 lanes.
template <int M>
__device__ __forceinline__ float join_over(float x, float y) {
  if constexpr (M == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else if constexpr (M == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    const bool up = lane_id() & M;
    constexpr int ctrl = M == 8 ? kDppRor8 : M == 4 ? kDppMirror8 : M == 2 ? kDppXor2 : kDppXor1;
    return (up ? y : x) + dpp<ctrl>(up ? x : y);
  }
}
template <int M, int NV>
__device__ __forceinline__ void join_all(float* x, const float* y) {
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = join_over<M>(x[i], y[i]);
}
// x[0 .. N) over the lane bits M, M / 2, ... (2 N = 2 M: bit 0 is left for a plain sum): value k's total ends up
// in the lanes whose bits from M down spell k.
template <int M, int N>
__device__ __forceinline__ float join_values(float* x) {
  static_assert(N == M || N == 1, "one lane bit per halving, and bit 0");
  if constexpr (N == 1) return x[0] + dpp<kDppXor1>(x[0]);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) x[i] = join_over<M>(x[i], x[i + N / 2]);
  return join_values<M / 2, N / 2>(x);
}

// One workgroup per (b, segment, channel block), NW waves with SW states each of the same 64 channels.
// A sub-chunk's per-channel values (dt, dt u, v) are formed once, a share of the tokens per wave, and
// passed through LDS with its rows of B and C; each wave's sums over its states come back the same
// way. Tokens behind the sequence are passed over as tokens of no step and no gradient.
template <class T, int S>
__global__ __launch_bounds__(64 * Bwd<S>::NW, S <= 16 ? 3 : 2) void scan_bwd(ScanArgs a, Plan p, BwdBufs w) {
  constexpr int SW = Bwd<S>::SW, NW = Bwd<S>::NW, kSub = Bwd<S>::kSub, kThreads = 64 * NW;
  constexpr int TW = kSub / NW;          // tokens a wave prepares and finishes
  constexpr int NV = 2 * SW;             // sums for dB and dC per token
  constexpr int RB = 32 / NV;            // tokens whose sums are joined together
  constexpr int EW = (kSub * S + kThreads - 1) / kThreads;  // elements of B a thread passes on
  static_assert(kSub % NW == 0 && kSub % RB == 0, "sub-chunk shares");
  __shared__ float s_dt[kSub][64], s_dtu[kSub][64], s_v[kSub][64];
  __shared__ float s_u[kSub][64], s_g[kSub][64], s_z[kSub][64], s_dy[kSub][64];  // for the end of the sub-chunk
  __shared__ float s_y[NW][kSub][64], s_q[NW][kSub][64], s_r[NW][kSub][64];
  __shared__ __align__(16) float s_b[kSub][S], s_c[kSub][S];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const Unit un = unit_of(blockIdx.x, p, a.C, a.G);
  const int C = a.C, N = a.N, c = un.c, s0 = wave * SW;
  const int n = length_of(a.lengths, un.b, N);
  const int t0 = un.seg * p.T, t1 = min(N, t0 + p.T), te = min(t1, n);
  const long long row0 = (long long)un.b * N;
  const T* u = (const T*)a.u + row0 * a.us;
  const T* de = (const T*)a.delta + row0 * a.ds;
  const bool gate = a.z;
  const T* z = gate ? (const T*)a.z + row0 * a.zs : u;
  const long long zs = gate ? a.zs : a.us;
  const T* dy = (const T*)a.dy + row0 * C;
  const T* bm = (const T*)a.bm + row0 * a.bs + (long long)un.g * S;
  const T* cm = (const T*)a.cm + row0 * a.cs + (long long)un.g * S;
  const long long seg = (long long)un.b * p.nseg + un.seg;
  // The padding's sums are zeros: with its states, which may not be finite, they would be 0 times those.
  for (int t = max(te, t0); t < t1; ++t)
    if (l < 2 * SW) w.mats[((row0 + t) * p.cb + un.cb) * 2 * S + 2 * SW * wave + l] = 0.f;
  float A2[SW], hs[SW], q[SW], dA[SW];
  for (int s = 0; s < SW; ++s) {
    A2[s] = a.A[(long long)c * S + s0 + s] * kLog2e;
    // (Zeros where the sequence ends before: its states may not be finite, and meet gradients of 0 here.)
    const float start = w.ends[(seg * S + s0 + s) * C + c];
    hs[s] = t0 < te ? start : 0.f;
    q[s] = w.back[(seg * S + s0 + s) * C + c];  // a q of the token behind
    dA[s] = 0.f;
  }
  const float db = a.dbias ? a.dbias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  float dD = 0.f, ddb = 0.f;
  // A sub-chunk's inputs, loaded while the one behind it is worked on, without a branch (past the
  // segment: its last row again); what is no token's is zeroed when it is used.
  float nu[TW], nd[TW], nv[TW], nz[TW], nb[EW], nc[EW], nck[SW], npast;
  auto fetch = [&](int tc) {
    const uint32_t off = lane_part(c, sizeof(T)), off4 = lane_part(c, 4);
#pragma unroll
    for (int j = 0; j < TW; ++j) {
      const long long t = min(tc + wave * TW + j, t1 - 1);
      nu[j] = at(u + t * a.us, off);
      nd[j] = at(de + t * a.ds, off);
      nv[j] = at(dy + t * C, off);
      nz[j] = at(z + t * zs, off);
    }
#pragma unroll
    for (int i = 0; i < EW; ++i) {
      const int e = threadIdx.x + i * kThreads;
      const long long t = min(tc + e / S, t1 - 1);
      nb[i] = (float)bm[t * a.bs + e % S];
      nc[i] = (float)cm[t * a.cs + e % S];
    }
    const long long k = (long long)un.b * w.nsub + tc / kSub;
    npast = at(w.cksum + k * C, off4);
    for (int s = 0; s < SW; ++s) nck[s] = at(w.ck + (k * S + s0 + s) * C, off4);
  };
  // Where the lane's sum over the channels goes: its token of the RB and its place in that token's row.
  const int tok = RB == 4 ? (l >> 5 & 1) | (l >> 4 & 1) << 1 : l >> 5, k = l / 2 % NV;
  static_assert(RB == 4 || RB == 2, "token bits of a lane");
  const int mat_at = tok * p.cb * 2 * S + (k / SW) * S + s0 + k % SW;
  const int last = t0 + (t1 - 1 - t0) / kSub * kSub;
  fetch(last);
  for (int tc = last; tc >= t0; tc -= kSub) {
    float h0[SW];
#pragma unroll
    for (int j = 0; j < TW; ++j) {
      const int i = wave * TW + j;
      const bool in = tc + i < te && un.live;
      const float uu = in ? nu[j] : 0.f, g = in ? nv[j] : 0.f;
      float grad, dt = step_grad_of(nd[j] + db, a.softplus, grad);
      dt = in ? dt : 0.f;
      s_dt[i][l] = dt;
      s_dtu[i][l] = dt * uu;
      s_v[i][l] = gate && in ? g * (nz[j] * sigmoid(nz[j])) : g;
      s_u[i][l] = uu, s_g[i][l] = grad, s_z[i][l] = nz[j], s_dy[i][l] = g;
    }
#pragma unroll
    for (int i = 0; i < EW; ++i) {
      const int e = threadIdx.x + i * kThreads;
      const bool in = tc + e / S < te;
      if (kSub * S % kThreads == 0 || e < kSub * S) {
        (&s_b[0][0])[e] = in ? nb[i] : 0.f;
        (&s_c[0][0])[e] = in ? nc[i] : 0.f;
      }
    }
    for (int s = 0; s < SW; ++s) h0[s] = fmaf(exp2_hw(A2[s] * npast), hs[s], nck[s]);
    __syncthreads();
    if (tc > t0) fetch(tc - kSub);
    float e[kSub][SW], h[kSub][SW];
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      float bv[SW], cv[SW];
      load_params<SW>(&s_b[j][s0], bv);
      load_params<SW>(&s_c[j][s0], cv);
      const float dt = s_dt[j][l], dtu = s_dtu[j][l];
      float y = 0.f;
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        e[j][s] = exp2_hw(dt * A2[s]);
        h[j][s] = fmaf(e[j][s], j ? h[j ? j - 1 : 0][s] : h0[s], dtu * bv[s]);
        y = fmaf(cv[s], h[j][s], y);
      }
      s_y[wave][j][l] = y;  // (used with a gate; without a branch the tokens' work interleaves)
      if (j & 1) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int jb = kSub - RB; jb >= 0; jb -= RB) {
      // The sums over the channels are joined as the tokens come, so that few wait in registers.
      float x[NV], l0[NV], l1[NV];
#pragma unroll
      for (int jj = RB - 1; jj >= 0; --jj) {
        const int j = jb + jj;
        float bv[SW], cv[SW];
        load_params<SW>(&s_b[j][s0], bv);
        load_params<SW>(&s_c[j][s0], cv);
        const float dt = s_dt[j][l], dtu = s_dtu[j][l], v = s_v[j][l];
        float qb = 0.f, r = 0.f;
#pragma unroll
        for (int s = 0; s < SW; ++s) {
          q[s] = fmaf(v, cv[s], q[s]);
          x[s] = q[s] * dtu;
          x[SW + s] = v * h[j][s];
          qb = fmaf(q[s], bv[s], qb);
          q[s] *= e[j][s];
          const float g = q[s] * (j ? h[j ? j - 1 : 0][s] : h0[s]);
          r = fmaf(g, A2[s], r);
          dA[s] = fmaf(g, dt, dA[s]);
        }
        s_q[wave][j][l] = qb;
        s_r[wave][j][l] = r;
        if (jj & 1) {
          for (int i = 0; i < NV; ++i) l0[i] = x[i];
        } else {
          join_all<32, NV>(x, l0);
          if (RB == 4 && (jj & 2)) {
            for (int i = 0; i < NV; ++i) l1[i] = x[i];
          } else if (RB == 4) {
            join_all<16, NV>(x, l1);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const float total = join_values<NV, NV>(x);
      if (!(l & 1) && tc + jb + tok < te) put(w.mats + ((row0 + tc + jb) * p.cb + un.cb) * 2 * S, lane_part(mat_at, 4), total);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TW; ++j) {
      const int i = wave * TW + j, t = tc + i;
      if (t < t1 && un.live) {
        float du = 0.f, dd = 0.f, dz = 0.f;
        if (t < n) {
          float sq = 0.f, sr = 0.f, sy = 0.f;
          for (int k = 0; k < NW; ++k) sq += s_q[k][i][l], sr += s_r[k][i][l], sy += s_y[k][i][l];
          const float uu = s_u[i][l], v = s_v[i][l];
          du = fmaf(sq, s_dt[i][l], D * v);
          dd = fmaf(sq, uu, sr * kLn2) * s_g[i][l];  // (sr has A log2(e) for A)
          dD = fmaf(v, uu, dD);
          ddb += dd;
          if (gate) {
            const float zz = s_z[i][l], sg = sigmoid(zz);
            dz = s_dy[i][l] * fmaf(D, uu, sy) * sg * fmaf(zz, 1.f - sg, 1.f);
          }
        }
        const long long row = (row0 + t) * C;
        const uint32_t off = lane_part(c, sizeof(T));
        put((T*)a.du + row, off, du);
        put((T*)a.ddelta + row, off, dd);
        if (gate) put((T*)a.dz + row, off, dz);
      }
    }
  }
  float* part = w.part + seg * ((long long)S * C + 2 * C);
  if (un.live)
    for (int s = 0; s < SW; ++s) part[(long long)(s0 + s) * C + c] = dA[s];
  __syncthreads();
  s_dt[wave][l] = dD;
  s_dtu[wave][l] = ddb;
  __syncthreads();
  if (wave == 0 && un.live) {
    for (int k = 1; k < NW; ++k) dD += s_dt[k][l], ddb += s_dtu[k][l];
    part[(long long)S * C + c] = dD;
    part[(long long)S * C + C + c] = ddb;
  }
}

struct StoreScanGrads {
  float *dA, *dD, *ddb;
  int C, S;
  __device__ void operator()(int col, float v) const {
    const int s = col / C, c = col - s * C;
    if (s < S) dA[(long long)c * S + s] = v;
    else if (s == S) {
      if (dD) dD[c] = v;
    } else if (ddb) ddb[c] = v;
  }
};

// The sums that end the backward pass, in one launch: the first sum_blocks workgroups add the segments'
// dA, dD and ddbias, the others the channel blocks of a group for dB and dC, one thread per
// (b, n, matrix, g, s).
template <class T>
__global__ __launch_bounds__(kSumThreads) void scan_bwd_sums(const float* __restrict__ part, long long segs, int C,
                                                             int sum_blocks, StoreScanGrads out,
                                                             const float* __restrict__ mats, T* __restrict__ dB,
                                                             T* __restrict__ dC, long long rows, int G, int S,
                                                             int cbg) {
  const long long block = wide_block();
  if (block < sum_blocks) {
    column_sum_block(part, segs, S * C + 2 * C, (int)block, out);
    return;
  }
  const long long id = (block - sum_blocks) * kSumThreads + threadIdx.x;
  const int width = 2 * G * S;
  if (id >= rows * width) return;
  const long long row = id / width;
  const int r = (int)(id - row * width), which = r / (G * S), gs = r - which * G * S, g = gs / S, s = gs - g * S;
  const float* m = mats + ((row * G + g) * cbg * 2 + which) * S + s;
  // (64 blocks at a time: one after the other 16384 of them drift.)
  float acc = 0.f;
  for (int k0 = 0; k0 < cbg; k0 += 64) {
    float part = 0.f;
#pragma unroll 4
    for (int k = k0; k < min(k0 + 64, cbg); ++k) part += m[(long long)k * 2 * S];
    acc += part;
  }
  (which ? dC : dB)[row * G * S + gs] = (T)acc;
}

// Segments: at most `want` waves in all, and at least min_tokens and at most max_tokens each (which goes before
// `want`), a multiple of `unit` tokens.
Plan plan_of(int B, int N, int C, int G, int want, int min_tokens, int max_tokens, int unit) {
  Plan p;
  p.cbg = (C / G + 63) / 64;
  p.cb = p.cbg * G;
  const long long blocks = (long long)B * p.cb;
  long long nseg = want / blocks;
  const long long most = (N + min_tokens - 1) / min_tokens;
  if (nseg > most) nseg = most;
  // (kMostUnits: a launch has fewer than 2^32 threads. Calls that fit the memory stay far below it.)
  nseg = std::max(nseg, std::min(((long long)N + max_tokens - 1) / max_tokens, std::max(1ll, kMostUnits / blocks)));
  const long long T = ((N + nseg - 1) / nseg + unit - 1) / unit * unit;
  p.T = (int)T;
  p.nseg = (int)((N + T - 1) / T);
  return p;
}
// Of the segment lengths from p's to `longest`, in steps of `unit` tokens or a 32nd, the one whose units (one per
// segment and block of channels, `slots` of them at a time) take the fewest tokens in all, one round after the other.
Plan full_rounds(Plan p, int B, int N, int slots, int longest, int unit) {
  const long long blocks = (long long)B * p.cb;
  const int step = (p.T / 32 + unit) / unit * unit;
  long long best = -1;
  for (int T = p.T; T <= longest; T += step) {
    const int nseg = (N + T - 1) / T;
    const long long tokens = (blocks * nseg + slots - 1) / slots * std::min(T, N);
    if (best < 0 || tokens < best) best = tokens, p.T = T, p.nseg = nseg;
  }
  return p;
}

// Forward.
//
// One segment, and one launch, where a second run over the tokens costs more than it gives:
//  * sequences of at most 26 tokens and one more for every 5 blocks of channels (768 channels, bf16, 16 states; one
//    launch and three, us): 1 x 24 tokens 11.5, 14.0; 1 x 32 14.2, 14.0; 8 x 32 14.4, 16.6; 8 x 48 19.9, 17.3; 24 x 64 26, 33;
//    24 x 96 37, 35; 64 x 160 71, 79;
//  * as many blocks as keep the SIMDs busy by themselves, found at 2048 tokens of 768 channels in bf16 (one and three):
//       8 states   1536 blocks  873,  780     1728  883, 1008     from 1600
//      16          1248        1179, 1039     1344 1184, 1200     from 1300
//      32           672        1085,  965      768 1084, 1083     from  720
//      64           768        2358, 2014      864 2365, 2305     from  820
//    It is not a law of the states alone: at 512 tokens 32 states change over between 576 (266, 255) and 768 (266, 307) as
//    well, but 64 between 576 (546, 472) and 768 (548, 569), so that up to 820 blocks of short sequences take 4 % longer.
//
// Otherwise segments for a number of waves, since segments cost the fold's traffic and their start, and waves hide what a
// token waits for:
//  * three per SIMD, and up to six while segments stay longer than 64 tokens (16 states, bf16, three and six: 2 x 4096 x
//    768 68, 72; 4 x 8192 x 768 189, 183);
//  * four with lengths, whose sequences end early, and their waves with them (from one case, 3 x <= 1999 x 1000 x 32, fp32:
//    a tenth less than three);
//  * none shorter than 8 to 24 tokens by the root of the length, since the fold takes longer the more there are (16 states;
//    24, 12 and 8 tokens: 1 x 102 x 64 21, 16, 14; 2 x 333 x 193 23, 17, 17; 1 x 1024 x 768 28, 26, 31);
//  * up to half longer where that fills rounds of a wave on each SIMD (2 x 2048 x 768, without and with: 16 states 49, 44;
//    64 states 119, 108), none longer than kLongest.
Plan fwd_plan(const ScanArgs& a, int S) {
  const long long blocks = (long long)a.B * ((a.C / a.G + 63) / 64 * a.G);
  const bool once = a.N <= 26 + blocks / 5 || blocks >= (S <= 8 ? 1600 : S <= 16 ? 1300 : S <= 32 ? 720 : 820);
  if (once) return plan_of(a.B, a.N, a.C, a.G, 1, a.N, a.N, kTokens);
  const long long by_length = std::min(6 * kSimds, blocks * (a.N / 64));
  const int shortest = std::min(24, std::max(8, (int)(0.45 * sqrt((double)a.N))));
  const long long want = std::max(by_length, (a.lengths ? 4 : 3) * kSimds);
  const Plan p = plan_of(a.B, a.N, a.C, a.G, (int)want, shortest, kLongest, kTokens);
  return full_rounds(p, a.B, a.N, (int)kSimds, std::max(p.T, std::min(p.T + p.T / 2, kLongest)), kTokens);
}
// Backward. The walk's workgroups (S / 4 or, of wide states, S / 8 waves) come in rounds of as many as the CUs hold (12 waves a
// CU by its registers, 8 of wide states), and a round takes as long as its segments. So of the segment lengths from a
// shortest to twice that, the one whose rounds take the fewest tokens in all (8 x 1024 x 512 x 64: 22 segments of 48 tokens
// are 5.5 rounds, 363 us, 16 of 64 are 4, 319 us). The shortest is 16 tokens (2 x 333 x 193 x 8 28 us; 24 36, 32 43) or what 4096
// blocks' segments leave, 1536 of wide states, whose segments cost more in the fold and in partial sums (1536 and twice
// as many, 2 x 4096 x 768, bf16: 32 states 252, 275; 64 486, 537); the longest kLongest.
Plan bwd_plan(const ScanArgs& a, int S) {
  const Plan p = plan_of(a.B, a.N, a.C, a.G, S <= 16 ? 4096 : 1536, 16, kLongest, kBwdSub);
  const int slots = 256 * (S <= 8 ? 6 : S <= 16 ? 3 : S <= 32 ? 2 : 1);
  return full_rounds(p, a.B, a.N, slots, std::max(p.T, std::min(2 * p.T, kLongest)), kBwdSub);
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Lays the backward's buffers out in the workspace; returns its size.
size_t bwd_layout(const ScanArgs& a, int S, const Plan& p, char* ws, BwdBufs* w) {
  w->nsub = (a.N + kBwdSub - 1) / kBwdSub;
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* r = reinterpret_cast<float*>(ws + at);
    at += align_up(floats * sizeof(float));
    return r;
  };
  const size_t B = a.B, C = a.C, segs = B * p.nseg, subs = B * w->nsub;
  w->ends = take(segs * S * C);
  w->back = take(segs * S * C);
  w->sums = take(segs * C);
  w->ck = take(subs * S * C);
  w->cksum = take(subs * C);
  w->mats = take(B * a.N * p.cb * 2 * S);
  w->part = take(segs * (S * C + 2 * C));
  return at;
}

hipError_t fold(const ScanArgs& a, int S, const Plan& p, float* ends, float* back, const float* sums, hipStream_t st) {
  const dim3 grid((unsigned)((a.C * S + kFoldThreads - 1) / kFoldThreads), (unsigned)a.B, back ? 2 : 1);
  hipLaunchKernelGGL(scan_fold, grid, dim3(kFoldThreads), 0, st, a.A, a.h0, ends, back, sums, a.dh0, a.C, S, p.nseg);
  return hipGetLastError();
}

template <class T, int S>
hipError_t fwd(const ScanArgs& a, void* ws, hipStream_t st) {
  const Plan p = fwd_plan(a, S);
  const long long units = (long long)a.B * p.nseg * p.cb;
  if (units > 0x7fffffffll) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((units + kWaves - 1) / kWaves)), block(64 * kWaves);
  float* ends = static_cast<float*>(ws);
  float* sums = ends + (size_t)a.B * p.nseg * S * a.C;
  if (p.nseg > 1) {
    hipLaunchKernelGGL((scan_fwd<T, S, false>), grid, block, 0, st, a, p, (int)units, ends, sums);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = fold(a, S, p, ends, nullptr, sums, st);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((scan_fwd<T, S, true>), grid, block, 0, st, a, p, (int)units, ends, sums);
  return hipGetLastError();
}

template <class T, int S>
hipError_t step(const ScanArgs& a, hipStream_t st) {
  const long long threads = (long long)a.B * a.C * (S / 4);
  const dim3 grid = wide_grid((threads + 255) / 256);
  const bool vec = ((reinterpret_cast<uintptr_t>(a.h0) | reinterpret_cast<uintptr_t>(a.h_out) |
                     reinterpret_cast<uintptr_t>(a.A)) & 15u) == 0;
  if (vec) hipLaunchKernelGGL((scan_step<T, S, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((scan_step<T, S, false>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <class T, int S>
hipError_t bwd(const ScanArgs& a, void* ws, hipStream_t st) {
  constexpr int SB = S < 16 ? S : 16;
  const Plan p = bwd_plan(a, S);
  BwdBufs w;
  bwd_layout(a, S, p, static_cast<char*>(ws), &w);
  const long long units = (long long)a.B * p.nseg * p.cb;
  const long long ends_units = units * (S / SB);
  const long long mats = (long long)a.B * a.N * 2 * a.G * S;
  if (ends_units > 0x7fffffffll) return hipErrorInvalidValue;
  hipLaunchKernelGGL((scan_bwd_ends<T, S, SB>), dim3((unsigned)((ends_units + kWaves - 1) / kWaves)), dim3(64 * kWaves),
                     0, st, a, p, (int)ends_units, w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = fold(a, S, p, w.ends, w.back, w.sums, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((scan_bwd<T, S>), dim3((unsigned)units), dim3(64 * Bwd<S>::NW), 0, st, a, p, w);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int sum_blocks = column_sum_blocks(S * a.C + 2 * a.C);
  hipLaunchKernelGGL(scan_bwd_sums<T>, wide_grid(sum_blocks + (mats + kSumThreads - 1) / kSumThreads), dim3(kSumThreads),
                     0, st, w.part, (long long)a.B * p.nseg, a.C, sum_blocks, StoreScanGrads{a.dA, a.dD, a.ddbias, a.C, S},
                     w.mats, (T*)a.dbm, (T*)a.dcm, (long long)a.B * a.N, a.G, S, p.cbg);
  return hipGetLastError();
}

}  // namespace

bool scan_supported_s(int S) { return S == 8 || S == 16 || S == 32 || S == 64; }

size_t scan_workspace_bytes(bool, int B, int N, int C, int S, int G) {
  ScanArgs a{};
  a.B = B, a.N = N, a.C = C, a.G = G;
  const int any = 0;
  int nseg = fwd_plan(a, S).nseg;
  a.lengths = &any;  // (not read: the plan of a call with lengths may have more segments)
  nseg = std::max(nseg, fwd_plan(a, S).nseg);
  return nseg > 1 ? (size_t)B * nseg * (S + 1) * C * sizeof(float) : 0;
}

size_t scan_bwd_workspace_bytes(bool, int B, int N, int C, int S, int G) {
  ScanArgs a{};
  a.B = B, a.N = N, a.C = C, a.G = G;
  BwdBufs w;
  return bwd_layout(a, S, bwd_plan(a, S), nullptr, &w);
}

#define TTT_SCAN(fn, ...)                                               \
  switch (S) {                                                          \
    case 8: return bf16_io ? fn<bf16, 8>(__VA_ARGS__) : fn<float, 8>(__VA_ARGS__);    \
    case 16: return bf16_io ? fn<bf16, 16>(__VA_ARGS__) : fn<float, 16>(__VA_ARGS__); \
    case 32: return bf16_io ? fn<bf16, 32>(__VA_ARGS__) : fn<float, 32>(__VA_ARGS__); \
    case 64: return bf16_io ? fn<bf16, 64>(__VA_ARGS__) : fn<float, 64>(__VA_ARGS__); \
  }                                                                     \
  return hipErrorInvalidValue;

hipError_t scan_launch(bool bf16_io, int S, const ScanArgs& a, void* ws, hipStream_t st) { TTT_SCAN(fwd, a, ws, st) }
hipError_t scan_step_launch(bool bf16_io, int S, const ScanArgs& a, hipStream_t st) { TTT_SCAN(step, a, st) }
hipError_t scan_bwd_launch(bool bf16_io, int S, const ScanArgs& a, void* ws, hipStream_t st) { TTT_SCAN(bwd, a, ws, st) }
#undef TTT_SCAN

}  // namespace ttt
