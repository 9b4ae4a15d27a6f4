// Gated linear recurrence: forward, one token at a time, and backward. Per channel,
//   la = -scale softplus(lam) sigmoid(r),  a = exp(la),  m = sqrt(1 - a^2),  h = a h + m sigmoid(i) x,  y = h.
// Backward, with q_n = dy_n + a_{n+1} q_{n+1}:
//   dx = q m sig(i),  di = q m x sig(i) (1 - sig(i)),  t = q (a la h_{n-1} - a^2 (la / m) sig(i) x),
//   dr = t (1 - sig(r)),  dlam = sum t sig(lam) / softplus(lam),  dh0 = a_0 q_0.
// t is la times the gradient of la: m's derivative -a^2 / m is infinite where a is 1, but la / m goes to 0 there
// with the root of la.
//
// Over a run of tokens h goes to A h + e, A the product of the decays and e the end from zero; two runs, one behind the other, are
// (A2 A1, A2 e1 + e2). So a sequence is cut into tiles of W waves x TW tokens x 64 V channels that run at once, and every input is read
// and every output written once: a tile loads its tokens and forms their a and m sigmoid(i) x in registers, joins its waves' pairs in LDS,
// tells the other tiles its own, folds those of the tiles before it onto the last state that is known, and walks its tokens again from
// registers (a single-pass scan with decoupled look-back, as Merrill and Garland published it in 2016; it is a method here, the code is
// written for this recurrence). The way back does the same from the sequences' ends on for q, with the states that the forward pass kept at every
// 64th token for h. Sums over tokens (lam's) are written for each tile and added in a fixed order; folds are in the tokens' order whatever
// comes first, so that the same call gives the same bits.
//
// Bound by HBM, then by the vector ALU: 32 instructions an element forward, 72 backward, five of which (two
// exponentials, two reciprocals, a root) take four times as long. 4 x 8192 x 768 in bf16, slow decays (of 0.78 a token and slower, Gates): forward
// 52 us (201 MB, 3.9 TB/s; the bytes alone 39), 4647 with a thread a channel and no tiles; backward 100 us (352 MB, 3.5 TB/s; the bytes 68,
// the ALU busy for 49). With a fast decay in every wave, or fast ones alone, 3 us more each. As many tokens in sequences of one tile, which tell and
// ask for nothing, take 39 us forward (256 x 128 x 768) and 78 backward (512 x 64 x 768); clearing the board is 3 of the rest.
#include <type_traits>

#include "internal.hpp"
#include "lm.hpp"
#include "rowops.hpp"

namespace ttt {
namespace {

constexpr int kThreads = 64;  // of a step's workgroup

// (exp(u) - 1) / u for -1/2 <= u <= 0, within 1.1 * 2^-24 of it (a polynomial through Chebyshev's nodes), and 1 - exp(u) for
// u <= 0: by that where the difference would lose bits; e is exp(u).
__device__ __forceinline__ float expm1_part(float u) {
  float p = 0.0011237150756642222f;
  p = fmaf(p, u, 0.008190003223717213f);
  p = fmaf(p, u, 0.04163024201989174f);
  p = fmaf(p, u, 0.16666245460510254f);
  p = fmaf(p, u, 0.4999998211860657f);
  return fmaf(p, u, 1.f);
}
__device__ __forceinline__ float one_minus(float u, float e) { return u > -0.5f ? -u * expm1_part(u) : 1.f - e; }
__device__ __forceinline__ float root(float v) { return __builtin_amdgcn_sqrtf(v); }

// log(1 + exp(v)): exp(-|v|) from its base-2 exponent in two parts (as one it would lose 2 |v| 2^-24 of itself), log1p(e) = s P(s^2)
// with s = e / (2 + e), P within 1.6e-8, which is 8e-9 of it, over e in (0, 1].
__device__ __forceinline__ float softplus(float v) {
  const float w = fmaxf(-fabsf(v), -200.f), hi = w * kLog2e;
  const float lo = fmaf(w, kLog2e, -hi) + w * 1.925962991e-8f;  // (log2(e) less kLog2e)
  const float e = exp2_hw(hi) * fmaf(lo, 0.69314718f, 1.f);
  const float s = e / (2.f + e), q = s * s;
  float p = 0.2817465662956238f;
  p = fmaf(p, q, 0.2796141803264618f);
  p = fmaf(p, q, 0.40024852752685547f);
  p = fmaf(p, q, 0.6666631698608398f);
  p = fmaf(p, q, 2.f);
  return v == v ? fmaf(s, p, fmaxf(v, 0.f)) : v;
}

// k = scale softplus(lam) is the decay's largest exponent. Where it is at most kSmall for a whole wave, as ordinary decays are (0.78 a
// token and slower), E = a - 1 is la times a polynomial (within 5e-9), a = 1 + E and 1 - a^2 = -E (2 + E), without an
// exponential or a choice; `wide` says that it is not.
constexpr float kSmall = 0.25f;

struct Gates {
  float gr, gi, la, a, w;  // sigmoid(r), sigmoid(i), log a, a, 1 - a^2
  __device__ __forceinline__ Gates(float r, float i, float k, bool wide) {
    gr = sigmoid(r), gi = sigmoid(i);
    la = -k * gr;
    if (wide) {
      a = exp2_hw(kLog2e * la);
      w = one_minus(2.f * la, a * a);
    } else {
      float p = 0.007514301221817732f;
      p = fmaf(p, la, 0.04149100184440613f);
      p = fmaf(p, la, 0.16665112972259521f);
      p = fmaf(p, la, 0.4999995231628418f);
      const float E = la * fmaf(p, la, 1.f);
      a = 1.f + E;
      w = -E * (2.f + E);
    }
  }
};
// A condition that is the same for the whole wave, as the compiler cannot tell.
__device__ __forceinline__ bool uniform(bool v) { return __builtin_amdgcn_readfirstlane(v ? 1 : 0) != 0; }

__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

// A lane's part of a row that is the same for the whole wave: the row's address stays in SGPRs, the lane's offset in one 32-bit
// register. (The empty asm keeps the two apart: added up they would be a 64-bit address per lane and row.)
__device__ __forceinline__ uint32_t lane_part(int c, int size) {
  uint32_t off = (uint32_t)c * (uint32_t)size;
  asm volatile("" : "+v"(off));
  return off;
}

// V neighbouring channels of one token as they are loaded (V = 2: 4 or 8 bytes, at any alignment of the elements), and stores of them.
template <class T, int V>
struct Pair {
  typedef typename std::conditional<sizeof(T) * V == 8, uint2, typename std::conditional<sizeof(T) * V == 4, uint32_t, uint16_t>::type>::type Bits;
  Bits b;
  __device__ __forceinline__ void load(const T* row, uint32_t off) {
    typedef Bits Any __attribute__((aligned(sizeof(T))));
    b = *reinterpret_cast<const Any*>(reinterpret_cast<const char*>(row) + off);
  }
  // To be looked at anew.
  __device__ __forceinline__ void hide() {
    if constexpr (sizeof(Bits) == 8) asm volatile("" : "+v"(b.x), "+v"(b.y));
    else asm volatile("" : "+v"(b));
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(Bits) == 8) return __uint_as_float(i ? b.y : b.x);
    else if constexpr (sizeof(T) == 4) return __uint_as_float(b);
    else return __uint_as_float(i ? (uint32_t)b & 0xffff0000u : (uint32_t)b << 16);
  }
  static __device__ __forceinline__ void store(T* row, uint32_t off, const float* v) {
    asm volatile("" : "+v"(off));  // (in the store's own block, or the compiler keeps the offset as 64 bits and adds the row to it)
    char* p = reinterpret_cast<char*>(row) + off;
    if constexpr (V == 1) {
      *reinterpret_cast<T*>(p) = (T)v[0];
    } else if constexpr (sizeof(T) == 4) {
      typedef uint2 Any __attribute__((aligned(4)));
      *reinterpret_cast<Any*>(p) = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
    } else {
      typedef uint32_t Any __attribute__((aligned(2)));
      typedef __bf16 two __attribute__((ext_vector_type(2)));
      typedef float ftwo __attribute__((ext_vector_type(2)));
      *reinterpret_cast<Any*>(p) = __builtin_bit_cast(uint32_t, __builtin_convertvector(ftwo{v[0], v[1]}, two));
    }
  }
};

// ---- what tiles tell each other ---------------------------------------------------------------
// A tile of a column (64 V channels of a sequence) tells the later ones its (decay, end) pairs, and every kGroup-th its
// end state: 64-bit words that are all ones until they are there, written and read whole by device-scope atomics, so that a word
// says by itself that it has come. A NaN is told as the one NaN that is not all ones. (Groups of 8 and of 32 tiles are
// no faster.) A wait that exceeds kMostPolls, some seconds, gives NaN (a word that has not come reads as one): there is none without end.
constexpr int kGroup = 16;
constexpr unsigned long long kNotYet = ~0ull;
constexpr int kMostPolls = 1 << 22;

__device__ __forceinline__ uint32_t word_of(float v) { return v == v ? __float_as_uint(v) : 0x7fc00000u; }
__device__ __forceinline__ void tell(unsigned long long* p, float lo, float hi) {
  __hip_atomic_store(p, (unsigned long long)word_of(hi) << 32 | word_of(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long ask(const unsigned long long* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Words: the columns' ticket counters, then [tiles][channels] pairs and [groups][channels] states of every sequence.
struct Board {
  unsigned* tickets;
  unsigned long long *pairs, *states;
};
// Two boards, one behind the other, each with its tickets' words first; words in twos.
constexpr int kClearThreads = 256;
__global__ __launch_bounds__(kClearThreads) void clear_board(ulonglong2* p, long long tickets, long long second, long long tickets2,
                                                             long long words) {
  const long long k = wide_block() * kClearThreads + threadIdx.x, at = 2 * k;
  const bool ticket = at < tickets || (at >= second && at < second + tickets2);
  const unsigned long long v = ticket ? 0ull : kNotYet;
  if (at < words) p[k] = make_ulonglong2(v, v);
}

// A workgroup's tile: its column goes by its number, its place there by a ticket of the column's, drawn in the order in which workgroups
// start. A tile waits for tiles of smaller tickets alone: they have started and wait for still smaller ones, so that every wait
// ends. (A counter for each column, in a line of its own: from one for all, hundreds of workgroups at once take 4 us.)
constexpr int kTicketWords = 16;
struct Tile {
  int tile, b, column;
};
// False where there is no tile for this workgroup.
__device__ __forceinline__ bool draw(const Board& board, int tiles, int columns, unsigned total, Tile& k) {
  const unsigned id = (unsigned)wide_block();
  if (id >= total) return false;
  const unsigned all = total / (unsigned)tiles;  // columns of all sequences
  const unsigned of = id % all;
  k.b = (int)(of / (unsigned)columns), k.column = (int)(of - (unsigned)k.b * (unsigned)columns);
  k.tile = 0;
  if (tiles > 1) {
    __shared__ unsigned drawn;
    if (threadIdx.x == 0) drawn = atomicAdd(board.tickets + (long long)of * (2 * kTicketWords), 1u);
    __syncthreads();
    k.tile = __builtin_amdgcn_readfirstlane(drawn);
  }
  return true;
}

// K times V neighbouring words, `step` apart, the first `count` of them asked for until they have come: all at once, and again only
// those that had not.
template <int K, int V>
__device__ __forceinline__ void ask_all(unsigned long long (&v)[K][V], const unsigned long long* p, long long step, int count) {
#pragma unroll
  for (int q = 0; q < K; ++q)
    for (int i = 0; i < V; ++i) v[q][i] = q < count ? kNotYet : 0;
  for (int polls = 0; polls < kMostPolls; ++polls) {
    bool there = true;
#pragma unroll
    for (int q = 0; q < K; ++q)
      for (int i = 0; i < V; ++i)
        if (v[q][i] == kNotYet) v[q][i] = ask(p + q * step + i);
#pragma unroll
    for (int q = 0; q < K; ++q)
      for (int i = 0; i < V; ++i) there = there && v[q][i] != kNotYet;
    if (__all(there)) return;
    __builtin_amdgcn_s_sleep(1);
  }
}
__device__ __forceinline__ float2 pair_of(unsigned long long w) {
  return make_float2(__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32)));
}

// What the waves of a workgroup share.
template <int W, int CH>
struct Desk {
  float2 part[W][CH], back[kGroup][CH];
  float begin[CH];
};

// Board, LDS and registers: see the file's head. The tokens' decays and inputs stay in registers between the two walks (126 of them with
// two channels a lane and 16 tokens, two workgroups a CU); all loads of a tile are under way at once, and the other workgroup's
// computation covers them. (Workgroups that stay and load their next tile while they wait: 66 us and more, since the loads before the
// wait are waited for with the words that are asked for.)
template <class T, int W, int V, int TW>
__global__ __launch_bounds__(64 * W) void recurrence_fwd(RecurrenceArgs a, int tiles, int columns, unsigned total, Board board) {
  constexpr int TILE = TW * W, CH = 64 * V;
  __shared__ Desk<W, CH> desk;
  Tile k;
  if (!draw(board, tiles, columns, total, k)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, C = a.C, N = a.N;
  const int wide = columns * CH, rows = (N + kKept - 1) / kKept;
  const int c0 = k.column * CH + lane * V, c = min(c0, C - V);  // (past the last channel the last ones again: an odd last channel's lane has the one before it too, of the same wave, with the same results)
  const bool mine = c0 < C;
  const int n = length_of(a.lengths, k.b, N), t0 = k.tile * TILE + wave * TW;
  const int live = n - t0, inside = N - t0;  // tokens of this run and those behind it, of the sequence and of the padded one
  const long long row = (long long)k.b * N + t0;
  const uint32_t off = lane_part(c, sizeof(T));
  T* py = a.y ? (T*)a.y + row * C : nullptr;
  if (k.tile * TILE >= n && k.tile > 0) {  // nothing but padding
    const float o[V] = {};
    if (py && mine)
      for (int t = 0; t < min(TW, inside); ++t) Pair<T, V>::store(py, off, o), py += C;
    return;
  }
  float kk[V];  // (first: loads come back in order)
  for (int i = 0; i < V; ++i) kk[i] = a.lam[c + i];
  Pair<T, V> x[TW], r[TW], g[TW];
  const int from = min(t0, N - 1);  // (past the last token: the last again)
  const T *px = (const T*)a.x + ((long long)k.b * N + from) * a.xs, *pr = (const T*)a.r + ((long long)k.b * N + from) * a.rs;
  const T* pi = (const T*)a.i + ((long long)k.b * N + from) * a.is;
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    x[t].load(px, off), r[t].load(pr, off), g[t].load(pi, off);
    if (t + 1 < inside) px += a.xs, pr += a.rs, pi += a.is;
  }
  bool far = false;
  for (int i = 0; i < V; ++i) kk[i] = a.scale * softplus(kk[i]), far = far || kk[i] > kSmall;
  // (Of a run without padding and steep decays the tokens are one straight piece of code.)
  const bool steep = uniform(__any(far)), plain = uniform(live >= TW && !steep);
  float A[V], e[V], av[TW][V], bv[TW][V];
  for (int i = 0; i < V; ++i) A[i] = 1.f, e[i] = 0.f;
  auto all = [&](auto plain) {
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      if (plain.value || t < live) {
        for (int i = 0; i < V; ++i) {
          const Gates q(r[t].get(i), g[t].get(i), kk[i], !plain.value && steep);
          av[t][i] = q.a;
          bv[t][i] = root(q.w) * q.gi * x[t].get(i);
          A[i] *= av[t][i];
          e[i] = fmaf(av[t][i], e[i], bv[t][i]);
        }
      } else {
        for (int i = 0; i < V; ++i) av[t][i] = 1.f, bv[t][i] = 0.f;
      }
    }
  };
  if (plain) all(std::true_type{});
  else all(std::false_type{});
  for (int i = 0; i < V; ++i) desk.part[wave][lane * V + i] = make_float2(A[i], e[i]);
  __syncthreads();
  float pa[V], pe[V];  // the pair of the waves before this one; with the last's own, the tile's
  for (int i = 0; i < V; ++i) pa[i] = 1.f, pe[i] = 0.f;
  for (int w = 0; w < wave; ++w)
    for (int i = 0; i < V; ++i) {
      const float2 p = desk.part[w][lane * V + i];
      pa[i] *= p.x, pe[i] = fmaf(p.x, pe[i], p.y);
    }
  const int group = k.tile / kGroup, count = k.tile - group * kGroup;  // tiles of its group before this one
  if (count > 0 || wave == W - 1) {
    float ta[V], te[V], h[V];
    for (int i = 0; i < V; ++i) ta[i] = pa[i] * A[i], te[i] = fmaf(A[i], pe[i], e[i]);
    unsigned long long* pairs = board.pairs + ((long long)k.b * tiles + group * kGroup) * wide + k.column * CH + lane * V;
    unsigned long long* states =
        board.states + ((long long)k.b * ((tiles + kGroup - 1) / kGroup) + group) * wide + k.column * CH + lane * V;
    if (wave == W - 1 && k.tile < tiles - 1)
      for (int i = 0; i < V; ++i) tell(pairs + (long long)count * wide + i, ta[i], te[i]);
    // A wave asks for the pairs of an equal run of the group's tiles, and the last wave, whose run ends with the group, for the state
    // before it.
    constexpr int EACH = kGroup / W;
    static_assert(kGroup % W == 0, "");
    const int first = wave * EACH;
    if (first < count) {
      unsigned long long v[EACH][V];
      ask_all(v, pairs + (long long)first * wide, wide, count - first);
#pragma unroll
      for (int q = 0; q < EACH; ++q)
        for (int i = 0; i < V; ++i) desk.back[first + q][lane * V + i] = pair_of(v[q][i]);
    }
    if (wave == W - 1) {
      unsigned long long v[1][V];
      if (group > 0) ask_all(v, states - wide, wide, 1);
      for (int i = 0; i < V; ++i) h[i] = group > 0 ? pair_of(v[0][i]).x : a.h0 ? a.h0[(long long)k.b * C + c + i] : 0.f;
    }
    if (count > 0) __syncthreads();
    if (wave == W - 1) {
      for (int j = 0; j < count; ++j)
        for (int i = 0; i < V; ++i) {
          const float2 p = desk.back[j][lane * V + i];
          h[i] = fmaf(p.x, h[i], p.y);
        }
      for (int i = 0; i < V; ++i) {
        desk.begin[lane * V + i] = h[i];
        h[i] = fmaf(ta[i], h[i], te[i]);
        if (count == kGroup - 1 && k.tile < tiles - 1) tell(states + i, h[i], 0.f);
      }
      if (mine && (k.tile + 1) * TILE >= n)
        for (int i = 0; i < V; ++i) {
          if (a.h_out) a.h_out[(long long)k.b * C + c + i] = h[i];
          if (a.states)  // before padding's tokens in later tiles: the last
            for (int j = ((k.tile + 1) * TILE + kKept - 1) / kKept; j < rows; ++j)
              a.states[((long long)k.b * rows + j) * C + c + i] = h[i];
        }
    }
  }
  __syncthreads();
  if (!mine || inside <= 0) return;
  float h[V];
  for (int i = 0; i < V; ++i) h[i] = fmaf(pa[i], desk.begin[lane * V + i], pe[i]);
  if (a.states && t0 % kKept == 0)
    for (int i = 0; i < V; ++i) a.states[((long long)k.b * rows + t0 / kKept) * C + c + i] = h[i];
  if (!py) return;
  auto put = [&](auto plain) {
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      float o[V];
      for (int i = 0; i < V; ++i) h[i] = fmaf(av[t][i], h[i], bv[t][i]), o[i] = plain.value || t < live ? h[i] : 0.f;
      if (plain.value || t < inside) Pair<T, V>::store(py, off, o);
      py += C;
    }
  };
  if (plain) put(std::true_type{});
  else put(std::false_type{});
}

// A channel of a sequence a thread: 64 x 1536 in bf16 take 2.7 us, a launch's start and end.
template <class T>
__global__ __launch_bounds__(kThreads) void recurrence_step(RecurrenceArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y, C = a.C;
  if (c >= C) return;
  const Gates g((float)((const T*)a.r)[b * a.rs + c], (float)((const T*)a.i)[b * a.is + c], a.scale * softplus(a.lam[c]), true);
  const long long at = (long long)b * C + c;
  const float h = fmaf(g.a, a.h0[at], root(g.w) * g.gi * (float)((const T*)a.x)[b * a.xs + c]);
  ((T*)a.y)[at] = (T)h;
  a.h_out[at] = h;
}

// ---- backward ----------------------------------------------------------------------------------
template <int W, int CH>
struct DeskBack {
  float2 part[W][CH], back[kGroup][CH];
  float z[W][CH];  // what flows out of a wave's front where nothing flows in at its end; later, its sum of t
  float begin[CH];
};

// Tiles from the sequences' ends on. Fewer tokens a wave than forward, since five numbers a token stay in registers (16 waves of 4 tokens in
// bf16 instead of 8 of 8: 131 us; with twice the waves a CU, which then spill, 143). The decays' first walk gives the tile's (A, e), from
// which its tokens' h follow, and with it what flows out of its front where nothing flows in at its end.
template <class T, int W, int V, int TW>
__global__ __launch_bounds__(64 * W) void recurrence_bwd(RecurrenceArgs a, int tiles, int columns, unsigned total, Board board,
                                                              float* sums) {
  constexpr int TILE = TW * W, CH = 64 * V;
  __shared__ DeskBack<W, CH> desk;
  static_assert(TILE % kKept == 0, "a tile starts at a kept state");
  Tile k;
  if (!draw(board, tiles, columns, total, k)) return;
  k.tile = tiles - 1 - k.tile;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, C = a.C, N = a.N;
  const int wide = columns * CH, rows = (N + kKept - 1) / kKept;
  const int c0 = k.column * CH + lane * V, c = min(c0, C - V);  // (past the last channel the last ones again: an odd last channel's lane has the one before it too, of the same wave, with the same results)
  const bool mine = c0 < C;
  const int n = length_of(a.lengths, k.b, N), t0 = k.tile * TILE + wave * TW;
  const int live = n - t0, inside = N - t0;  // tokens of this run and those behind it, of the sequence and of the padded one
  const uint32_t off = lane_part(c, sizeof(T));
  const long long end = ((long long)k.b * N + t0 + TW - 1) * C;  // the run's last token
  T *ox = (T*)a.dx + end, *orr = (T*)a.dr + end, *oi = (T*)a.di + end;
  if (k.tile * TILE >= n && k.tile > 0) {  // nothing but padding
    const float o[V] = {};
    if (!mine) return;
    for (int t = TW - 1; t >= 0; --t) {
      if (t < inside) Pair<T, V>::store(ox, off, o), Pair<T, V>::store(orr, off, o), Pair<T, V>::store(oi, off, o);
      ox -= C, orr -= C, oi -= C;
    }
    if (wave == 0)
      for (int i = 0; i < V; ++i) sums[((long long)k.b * tiles + k.tile) * C + c + i] = 0.f;
    return;
  }
  float h[V], kk[V];  // (first: loads come back in order)
  for (int i = 0; i < V; ++i) {
    kk[i] = a.lam[c + i];
    h[i] = a.kept[((long long)k.b * rows + k.tile * TILE / kKept) * C + c + i];
  }
  Pair<T, V> x[TW], r[TW], g[TW], dy[TW];
  const long long from = (long long)k.b * N + min(t0, N - 1);  // (past the last token: the last again)
  const T *px = (const T*)a.x + from * a.xs, *pr = (const T*)a.r + from * a.rs, *pi = (const T*)a.i + from * a.is;
  const T* pd = (const T*)a.dy + from * C;
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    x[t].load(px, off), r[t].load(pr, off), g[t].load(pi, off), dy[t].load(pd, off);
    if (t + 1 < inside) px += a.xs, pr += a.rs, pi += a.is, pd += C;
  }
  bool far = false;
  for (int i = 0; i < V; ++i) kk[i] = a.scale * softplus(kk[i]), far = far || kk[i] > kSmall;
  const bool steep = uniform(__any(far));
  // Of a token: a; m sigmoid(i); x (1 - sigmoid(i)); t / q = a la (h - (a / m) sigmoid(i) x), at first what is taken from h; sigmoid(r).
  float av[TW][V], cx[TW][V], ci[TW][V], ct[TW][V], gr[TW][V];
  float A[V], e[V], z[V];
  for (int i = 0; i < V; ++i) A[i] = 1.f, e[i] = z[i] = 0.f;
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    if (t < live) {
      for (int i = 0; i < V; ++i) {
        const Gates q(r[t].get(i), g[t].get(i), kk[i], steep);
        const float inv = q.w < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(q.w);  // 1 / m; (m = 0 below the root's range)
        const float xv = x[t].get(i), m = q.w * inv, drive = q.gi * xv;
        av[t][i] = q.a;
        cx[t][i] = m * q.gi;
        ci[t][i] = xv * (1.f - q.gi);
        ct[t][i] = q.a * inv * drive;
        gr[t][i] = q.gr;
        A[i] *= q.a;
        e[i] = fmaf(q.a, e[i], m * drive);
      }
    } else {
      for (int i = 0; i < V; ++i) av[t][i] = 1.f, cx[t][i] = ci[t][i] = ct[t][i] = gr[t][i] = 0.f;
    }
  }
#pragma unroll
  for (int t = TW - 1; t >= 0; --t)
    for (int i = 0; i < V; ++i) z[i] = av[t][i] * ((t < live ? dy[t].get(i) : 0.f) + z[i]);
  // (x and dy stay as they were loaded.)
#pragma unroll
  for (int t = 0; t < TW; ++t) x[t].hide(), dy[t].hide();
  for (int i = 0; i < V; ++i) desk.part[wave][lane * V + i] = make_float2(A[i], e[i]), desk.z[wave][lane * V + i] = z[i];
  __syncthreads();
  // The tile's pair, told by the last wave as soon as it is there; the state before this wave's tokens, the pair of the waves behind it.
  const int group = k.tile / kGroup, last = n > 0 ? (n - 1) / TILE : 0;  // the sequence's last tile
  const int count = min(group * kGroup + kGroup - 1, last) - k.tile;     // tiles of its group behind this one
  const bool further = (group + 1) * kGroup <= last;
  unsigned long long* pairs = board.pairs + ((long long)k.b * tiles + k.tile) * wide + k.column * CH + lane * V;
  unsigned long long* states =
      board.states + ((long long)k.b * ((tiles + kGroup - 1) / kGroup) + group) * wide + k.column * CH + lane * V;
  float ta[V], tz[V];
  if (wave == W - 1) {
    for (int i = 0; i < V; ++i) ta[i] = 1.f, tz[i] = 0.f;
    for (int w = W - 1; w >= 0; --w)
      for (int i = 0; i < V; ++i) {
        const float p = desk.part[w][lane * V + i].x;
        ta[i] *= p, tz[i] = fmaf(p, tz[i], desk.z[w][lane * V + i]);
      }
    if (k.tile % kGroup != 0)
      for (int i = 0; i < V; ++i) tell(pairs + i, ta[i], tz[i]);
  }
  float pa[V], pz[V];
  for (int i = 0; i < V; ++i) pa[i] = 1.f, pz[i] = 0.f;
  for (int w = 0; w < wave; ++w)
    for (int i = 0; i < V; ++i) {
      const float2 p = desk.part[w][lane * V + i];
      h[i] = fmaf(p.x, h[i], p.y);
    }
  for (int w = W - 1; w > wave; --w)
    for (int i = 0; i < V; ++i) {
      const float p = desk.part[w][lane * V + i].x;
      pa[i] *= p, pz[i] = fmaf(p, pz[i], desk.z[w][lane * V + i]);
    }
#pragma unroll
  for (int t = 0; t < TW; ++t)
    for (int i = 0; i < V; ++i) {
      ct[t][i] = av[t][i] * (-kk[i] * gr[t][i]) * (h[i] - ct[t][i]);
      h[i] = fmaf(av[t][i], h[i], t < live ? cx[t][i] * x[t].get(i) : 0.f);
    }
  constexpr int EACH = kGroup / W;
  static_assert(kGroup % W == 0, "");
  const int first = wave * EACH;
  if (first < count) {
    unsigned long long v[EACH][V];
    ask_all(v, pairs + (long long)(first + 1) * wide, wide, count - first);
#pragma unroll
    for (int q = 0; q < EACH; ++q)
      for (int i = 0; i < V; ++i) desk.back[first + q][lane * V + i] = pair_of(v[q][i]);
  }
  float f[V];
  if (wave == W - 1) {
    unsigned long long v[1][V];
    if (further) ask_all(v, states + wide, wide, 1);
    for (int i = 0; i < V; ++i) f[i] = further ? pair_of(v[0][i]).x : 0.f;
  }
  if (count > 0) __syncthreads();
  if (wave == W - 1) {
    for (int j = count - 1; j >= 0; --j)
      for (int i = 0; i < V; ++i) {
        const float2 p = desk.back[j][lane * V + i];
        f[i] = fmaf(p.x, f[i], p.y);
      }
    for (int i = 0; i < V; ++i) {
      desk.begin[lane * V + i] = f[i];
      f[i] = fmaf(ta[i], f[i], tz[i]);
      if (k.tile % kGroup == 0 && k.tile > 0) tell(states + i, f[i], 0.f);
      if (k.tile == 0 && a.dh0 && mine) a.dh0[(long long)k.b * C + c + i] = f[i];
    }
  }
  __syncthreads();
  float sum[V] = {};
  for (int i = 0; i < V; ++i) z[i] = fmaf(pa[i], desk.begin[lane * V + i], pz[i]);
  if (mine) {
    auto put = [&](auto plain) {
#pragma unroll
      for (int t = TW - 1; t >= 0; --t) {
        float dx[V] = {}, dr[V] = {}, di[V] = {};
        if (plain.value || t < live)
          for (int i = 0; i < V; ++i) {
            const float q = dy[t].get(i) + z[i], l = q * ct[t][i];
            dx[i] = q * cx[t][i];
            di[i] = dx[i] * ci[t][i];
            dr[i] = l * (1.f - gr[t][i]);
            sum[i] += l;
            z[i] = av[t][i] * q;
          }
        if (plain.value || t < inside) Pair<T, V>::store(ox, off, dx), Pair<T, V>::store(orr, off, dr), Pair<T, V>::store(oi, off, di);
        ox -= C, orr -= C, oi -= C;
      }
    };
    if (uniform(live >= TW)) put(std::true_type{});
    else put(std::false_type{});
  }
  // (The z that flow out of the fronts have been read before the last barrier.)
  for (int i = 0; i < V; ++i) desk.z[wave][lane * V + i] = sum[i];
  __syncthreads();
  if (wave == 0 && mine)
    for (int i = 0; i < V; ++i) {
      float s = 0.f;
      for (int w = 0; w < W; ++w) s += desk.z[w][lane * V + i];
      sums[((long long)k.b * tiles + k.tile) * C + c + i] = s;
    }
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

// How a pass is cut up: W waves a workgroup, V channels a lane and TW tokens, tiles of a sequence, columns; the board's words, the
// tickets' among them, none where a sequence is one tile.
struct Plan {
  int W, V, TW, tiles, columns;
  long long words, tickets;
  long long workgroups(int B) const { return (long long)B * tiles * columns; }
};
Plan cut(int B, int N, int C, int W, int V, int TW) {
  Plan p{W, V, TW, (N + TW * W - 1) / (TW * W), (C + 64 * V - 1) / (64 * V), 0, 0};
  if (p.tiles == 1) return p;
  const long long columns = (long long)B * p.columns;
  p.tickets = columns * kTicketWords;
  p.words = p.tickets + columns * 64 * V * (p.tiles + (p.tiles + kGroup - 1) / kGroup);
  return p;
}
// Two channels a lane where that gives each CU a workgroup: a wave then moves 256 bytes (bf16) at a time and joins half as many pairs;
// otherwise one, for twice as many workgroups. One too where the last column would be a single channel: its lane would compute the channel
// before it, which another workgroup has, and the two may form their decays differently (Gates: by all of a
// column's channels): 4 x 8192 x 769 in bf16 70 us forward and 151 backward, x 770 62 and 123. (Tiles of 32 tokens
// for small calls gain a tenth at most, 1 x 512 x 256 8.5 -> 7.7 us, and lose where a sequence has many, 2 x 1024 x 768 11 -> 19.) As many
// tokens a lane as registers hold.
constexpr int kCus = 256;
template <class T>
Plan plan_of(int B, int N, int C, bool backward) {
  constexpr bool kHalf = sizeof(T) == 2;
  const int W = backward && !kHalf ? 16 : 8, TW = backward ? (kHalf ? 8 : 4) : (kHalf ? 16 : 8);
  const Plan two = cut(B, N, C, W, 2, TW);
  return C % 128 != 1 && two.workgroups(B) >= kCus ? two : cut(B, N, C, W, 1, TW);
}

Board board_of(const Plan& p, int B, unsigned long long* w) {
  unsigned long long* pairs = w + p.tickets;
  return Board{reinterpret_cast<unsigned*>(w), pairs, pairs + (long long)B * p.columns * 64 * p.V * p.tiles};
}

hipError_t clear(unsigned long long* w, const Plan& one, const Plan* two, hipStream_t st) {
  const long long words = one.words + (two ? two->words : 0);
  if (words == 0) return hipSuccess;
  hipLaunchKernelGGL(clear_board, wide_grid((words + 2 * kClearThreads - 1) / (2 * kClearThreads)), dim3(kClearThreads), 0, st,
                     reinterpret_cast<ulonglong2*>(w), one.tickets, one.words, two ? two->tickets : 0, words);
  return hipGetLastError();
}

template <class T, int W, int V, int TW>
void forward(const RecurrenceArgs& a, const Plan& p, unsigned long long* w, hipStream_t st) {
  const unsigned total = (unsigned)p.workgroups(a.B);
  hipLaunchKernelGGL((recurrence_fwd<T, W, V, TW>), wide_grid(total), dim3(64 * W), 0, st, a, p.tiles, p.columns, total,
                     board_of(p, a.B, w));
}
template <class T, int W, int V, int TW>
void backward(const RecurrenceArgs& a, const Plan& p, unsigned long long* w, float* sums, hipStream_t st) {
  const unsigned total = (unsigned)p.workgroups(a.B);
  hipLaunchKernelGGL((recurrence_bwd<T, W, V, TW>), wide_grid(total), dim3(64 * W), 0, st, a, p.tiles, p.columns, total,
                     board_of(p, a.B, w), sums);
}

// (By plan_of's pieces.)
template <class T>
hipError_t run_forward(const RecurrenceArgs& a, const Plan& p, unsigned long long* w, hipStream_t st) {
  constexpr int TW = sizeof(T) == 2 ? 16 : 8;
  p.V == 2 ? forward<T, 8, 2, TW>(a, p, w, st) : forward<T, 8, 1, TW>(a, p, w, st);
  return hipGetLastError();
}
template <class T>
hipError_t run_backward(const RecurrenceArgs& a, const Plan& p, unsigned long long* w, float* sums, hipStream_t st) {
  constexpr int W = sizeof(T) == 2 ? 8 : 16, TW = sizeof(T) == 2 ? 8 : 4;
  p.V == 2 ? backward<T, W, 2, TW>(a, p, w, sums, st) : backward<T, W, 1, TW>(a, p, w, sums, st);
  return hipGetLastError();
}

template <class T>
size_t forward_bytes(int B, int N, int C) {
  return (size_t)plan_of<T>(B, N, C, false).words * 8;
}

// The backward pass's workspace: the boards of both passes, the tiles' sums, the states.
struct BackLayout {
  size_t sums, states, bytes;
};
template <class T>
BackLayout back_layout(int B, int N, int C, bool kept) {
  const Plan p = plan_of<T>(B, N, C, true);
  BackLayout l;
  l.sums = round_up((size_t)p.words * 8 + (kept ? 0 : forward_bytes<T>(B, N, C)), 256);
  l.states = l.sums + round_up((size_t)B * p.tiles * C * 4, 256);
  l.bytes = l.states + (kept ? 0 : (size_t)B * ((N + kKept - 1) / kKept) * C * 4);
  return l;
}

template <class T>
hipError_t forward_call(const RecurrenceArgs& a, void* ws, hipStream_t st) {
  const Plan p = plan_of<T>(a.B, a.N, a.C, false);
  unsigned long long* w = static_cast<unsigned long long*>(ws);
  const hipError_t e = clear(w, p, nullptr, st);
  return e == hipSuccess ? run_forward<T>(a, p, w, st) : e;
}

template <class T>
hipError_t backward_call(RecurrenceArgs a, void* ws, hipStream_t st) {
  const bool kept = a.kept != nullptr;
  const BackLayout l = back_layout<T>(a.B, a.N, a.C, kept);
  const Plan p = plan_of<T>(a.B, a.N, a.C, true), q = plan_of<T>(a.B, a.N, a.C, false);
  unsigned long long* w = static_cast<unsigned long long*>(ws);
  float* sums = reinterpret_cast<float*>(static_cast<char*>(ws) + l.sums);
  hipError_t e = clear(w, p, kept ? nullptr : &q, st);
  if (e != hipSuccess) return e;
  if (!kept) {  // the forward pass again, for its states alone
    a.states = reinterpret_cast<float*>(static_cast<char*>(ws) + l.states);
    a.kept = a.states;
    e = run_forward<T>(a, q, w + p.words, st);
    if (e != hipSuccess) return e;
  }
  e = run_backward<T>(a, p, w, sums, st);
  if (e != hipSuccess) return e;
  return column_sum_launch(sums, (long long)a.B * p.tiles, a.C, StoreDecayGrad{a.lam, a.dlam}, st);
}

}  // namespace

size_t recurrence_workspace_bytes(bool bf16_io, int B, int N, int C) {
  return bf16_io ? forward_bytes<bf16>(B, N, C) : forward_bytes<float>(B, N, C);
}

hipError_t recurrence_launch(bool bf16_io, const RecurrenceArgs& a, void* ws, hipStream_t st) {
  return bf16_io ? forward_call<bf16>(a, ws, st) : forward_call<float>(a, ws, st);
}

hipError_t recurrence_step_launch(bool bf16_io, const RecurrenceArgs& a, hipStream_t st) {
  if (bf16_io) hipLaunchKernelGGL(recurrence_step<bf16>, grid_of(a), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL(recurrence_step<float>, grid_of(a), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

size_t recurrence_bwd_workspace_bytes(bool bf16_io, int B, int N, int C, bool kept) {
  return bf16_io ? back_layout<bf16>(B, N, C, kept).bytes : back_layout<float>(B, N, C, kept).bytes;
}

hipError_t recurrence_bwd_launch(bool bf16_io, const RecurrenceArgs& a, void* ws, hipStream_t st) {
  return bf16_io ? backward_call<bf16>(a, ws, st) : backward_call<float>(a, ws, st);
}

}  // namespace ttt
