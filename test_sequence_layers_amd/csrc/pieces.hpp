// 16-byte pieces of rows of any alignment and width (rmsnorm.hip, dropout.hip).
#pragma once

#include <type_traits>

#include "rowops.hpp"

namespace ttt {

// 16 bytes of a row, at any alignment of its elements: the hardware takes them so, and rows of odd widths are read as fast as others
// (1537 x 1001 fp32 backward TIME).
template <class T>
constexpr int kPiece = 16 / (int)sizeof(T);
typedef uint32_t Words __attribute__((ext_vector_type(4)));
typedef Words WordsAt2 __attribute__((aligned(2)));
typedef Words WordsAt4 __attribute__((aligned(4)));
template <class T>
struct Piece {
  typedef typename std::conditional<sizeof(T) == 2, WordsAt2, WordsAt4>::type Any;
  static constexpr int V = kPiece<T>;
  Words w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Any*>(p); }
  // The last `count` elements, at the front, and zeros: of a piece that ends with a row, as the row's last part of a piece.
  __device__ __forceinline__ void keep_last(int count) {
    const int bits = (V - count) * 8 * (int)sizeof(T);
    const uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
    const uint64_t a = bits >= 64 ? hi >> (bits & 63) : lo >> bits | (bits ? hi << (64 - bits) : 0);
    const uint64_t b = bits >= 64 ? 0 : hi >> bits;
    w = Words{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
  }
  // The first `count` elements (the same for the whole wave), and zeros.
  __device__ __forceinline__ void load_some(const T* p, int count) {
    w = Words{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V - 1; ++i)
      if (i < count) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint((float)p[i]);
        else w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i & 1));
      }
  }
  __device__ __forceinline__ void widen(float* out) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) out[i] = __uint_as_float(w[i]);
      else out[2 * i] = __uint_as_float(w[i] << 16), out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<Any*>(p) = Words{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
      const bf16x8 o = cat8(to_bf16x4(f32x4{v[0], v[1], v[2], v[3]}), to_bf16x4(f32x4{v[4], v[5], v[6], v[7]}));
      *reinterpret_cast<Any*>(p) = __builtin_bit_cast(Words, o);
    }
  }
  static __device__ __forceinline__ void store_some(T* p, const float* v, int count) {
#pragma unroll
    for (int i = 0; i < V - 1; ++i)
      if (i < count) p[i] = (T)v[i];
  }
};

}  // namespace ttt
