// Dropout's random numbers: Philox 4x32 in 10 rounds (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as
// 1, 2, 3, SC'11), a function of a 64-bit key and a counter, so that the mask is computed wherever it is wanted and never
// stored. One evaluation gives 8 elements 16 bits each: 4 words a piece would take twice the multiplications, and
// 16 bits hold the probability to 2^-17. Ten rounds are 20 products of 32 bits to 64, about 17 lane operations an element.
#pragma once

#include "rowops.hpp"

namespace ttt {

// What a call drops by: the caller's {seed, offset} on the device, the least 16-bit number that is kept (0: everything
// is, and rng is not read), and what kept values are multiplied by.
struct Drop {
  const unsigned long long* rng;
  uint32_t least;
  float scale;
};

// 16-bit number j of 8: halves of the words, the lower first.
struct Random8 {
  uint32_t w[4];
  __device__ __forceinline__ bool kept(int j, uint32_t least) const {
    return (j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu) >= least;
  }
  // Bit j: number j is kept.
  __device__ __forceinline__ uint32_t mask(uint32_t least) const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m |= kept(j, least) ? 1u << j : 0u;
    return m;
  }
};

__device__ __forceinline__ Random8 random8(unsigned long long seed, unsigned long long counter) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const unsigned long long p0 = (unsigned long long)c0 * 0xD2511F53u, p1 = (unsigned long long)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return Random8{{c0, c1, c2, c3}};
}

// The masks of a row that L lanes hold in K accesses of V elements (element (k L + lane) V + i): bit i of bits[k]. `first` is
// the counter of the row's first 8 elements.
template <int L, int K, int V>
struct RowMask {
  static_assert(V == 8 || (V == 4 && L % 2 == 0), "");
  uint32_t bits[K];
  __device__ __forceinline__ void make(unsigned long long seed, unsigned long long first, uint32_t least, int lane) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const unsigned piece = (unsigned)(k * L + lane);
      if constexpr (V == 8) bits[k] = random8(seed, first + piece).mask(least);
      else bits[k] = random8(seed, first + (piece >> 1)).mask(least) >> (4 * (lane & 1));
    }
  }
  __device__ __forceinline__ bool kept(int k, int i) const { return (bits[k] >> i) & 1u; }
};

}  // namespace ttt
