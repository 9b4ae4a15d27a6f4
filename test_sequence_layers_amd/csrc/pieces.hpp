// 16-byte pieces of rows of any alignment and width (rmsnorm.hip, dropout.hip).
#pragma once

#include <type_traits>

#include "rowops.hpp"

namespace ttt {

// 16 bytes of a row, at any alignment of its elements: the hardware takes them so, and rows of odd widths cost little more than others
// (norm of 32768 rows in bf16: 36.8 us of 768 channels, 37.6 of 766, 38.8 of 767, 46 with the end of a row, and its weights, element by element).
template <class T>
constexpr int kPiece = 16 / (int)sizeof(T);
typedef uint32_t Words __attribute__((ext_vector_type(4)));
typedef Words WordsAt2 __attribute__((aligned(2)));
typedef Words WordsAt4 __attribute__((aligned(4)));
typedef uint32_t TwoWords __attribute__((ext_vector_type(2)));
typedef TwoWords TwoWordsAt2 __attribute__((aligned(2)));
typedef TwoWords TwoWordsAt4 __attribute__((aligned(4)));
typedef uint32_t WordAt2 __attribute__((aligned(2)));
template <class T>
struct Piece {
  typedef typename std::conditional<sizeof(T) == 2, WordsAt2, WordsAt4>::type Any;
  typedef typename std::conditional<sizeof(T) == 2, TwoWordsAt2, TwoWordsAt4>::type Two;
  typedef typename std::conditional<sizeof(T) == 2, WordAt2, uint32_t>::type One;
  static constexpr int V = kPiece<T>;
  Words w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Any*>(p); }
  // Of a row of `count` elements, fewer than V: they become the last here.
  __device__ __forceinline__ void load_last(const T* p, int count) {
    w = Words{0, 0, 0, 0};
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (i >= V - count) {
        const T v = p[count - V + i];
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v);
        else w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, v) << (16 * (i & 1));
      }
  }
  __device__ __forceinline__ void widen(float* out) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) out[i] = __uint_as_float(w[i]);
      else out[2 * i] = __uint_as_float(w[i] << 16), out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Words narrow(const float* v) {
    if constexpr (sizeof(T) == 4) return Words{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    else return __builtin_bit_cast(Words, cat8(to_bf16x4(f32x4{v[0], v[1], v[2], v[3]}), to_bf16x4(f32x4{v[4], v[5], v[6], v[7]})));
  }
  static __device__ __forceinline__ void store(T* p, const float* v) { *reinterpret_cast<Any*>(p) = narrow(v); }
  // The last `count` elements (of 1 .. V - 1, the same for the whole wave) to p, by the binary digits of the count.
  static __device__ __forceinline__ void store_last(T* p, const float* v, int count) {
    const Words q = narrow(v);
    const int bits = (V - count) * 8 * (int)sizeof(T);
    const uint64_t lo = (uint64_t)q[1] << 32 | q[0], hi = (uint64_t)q[3] << 32 | q[2];
    uint64_t a = bits >= 64 ? hi >> (bits & 63) : lo >> bits | hi << (64 - bits);
    if (count * (int)sizeof(T) & 8) {
      *reinterpret_cast<Two*>(p) = TwoWords{(uint32_t)a, (uint32_t)(a >> 32)};
      a = hi >> (bits & 63), p += 8 / sizeof(T);
    }
    if (count * (int)sizeof(T) & 4) {
      *reinterpret_cast<One*>(p) = (uint32_t)a;
      a >>= 32, p += 4 / sizeof(T);
    }
    if constexpr (sizeof(T) == 2) {
      if (count & 1) *reinterpret_cast<uint16_t*>(p) = (uint16_t)a;
    }
  }
};

}  // namespace ttt
