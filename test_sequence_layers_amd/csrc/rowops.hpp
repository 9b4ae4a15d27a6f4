// Device pieces shared by the block operators' kernels: element loads and stores of either I/O type,
// sums over groups of lanes, and the sum of partial rows that ends the parameters' gradients.
#pragma once

#include "device.hpp"

namespace ttt {

// V elements of T as they are loaded, in one access of 8 or 16 bytes or one element; widened to fp32 where
// they are used. (Widened where they are loaded, inside a branch, they would be waited for there.)
template <class T, int V>
struct Raw {
  static constexpr int W = V * (int)sizeof(T) / 4;
  static_assert(W == 2 || W == 4, "8 or 16 bytes");
  typedef uint32_t Words __attribute__((ext_vector_type(W)));
  Words r;
  __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const Words*>(p); }
  __device__ __forceinline__ void widen(float* out) const {
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 2) {
        out[2 * i] = __uint_as_float(r[i] << 16);
        out[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      } else {
        out[i] = __uint_as_float(r[i]);
      }
    }
  }
};
template <class T>
struct Raw<T, 1> {
  T r;
  __device__ __forceinline__ void load(const T* p) { r = p[0]; }
  __device__ __forceinline__ void widen(float* out) const { out[0] = (float)r; }
};
template <class T, int V>
__device__ __forceinline__ void load_row(const T* p, float* out) {
  Raw<T, V> r;
  r.load(p);
  r.widen(out);
}

template <class T, int V>
__device__ __forceinline__ void store_row(T* p, const float* v) {
  if constexpr (V == 1) {
    p[0] = (T)v[0];
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    *reinterpret_cast<bf16x4*>(p) = to_bf16x4(f32x4{v[0], v[1], v[2], v[3]});
  } else if constexpr (sizeof(T) == 2) {
    const bf16x8 o = cat8(to_bf16x4(f32x4{v[0], v[1], v[2], v[3]}), to_bf16x4(f32x4{v[4], v[5], v[6], v[7]}));
    st16(p, __builtin_bit_cast(uint4, o));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// V fp32 parameters; in the vector case p is 16-byte aligned.
template <int V>
__device__ __forceinline__ void load_params(const float* p, float* out) {
  if constexpr (V == 1) {
    out[0] = p[0];
  } else {
    for (int i = 0; i < V; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      out[i] = q.x; out[i + 1] = q.y; out[i + 2] = q.z; out[i + 3] = q.w;
    }
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xB1;     // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;     // quad_perm [2, 3, 0, 1]
constexpr int kDppMirror8 = 0x141;   // lane i of 8 reads lane 7 - i
constexpr int kDppMirror16 = 0x140;  // lane i of 16 reads lane 15 - i
constexpr int kDppRor8 = 0x128;      // lane i of 16 reads lane i ^ 8

// Sum over aligned groups of L lanes (L a power of two up to 64); every lane gets it. Within 16
// lanes by DPP: once the lanes of a quad agree, the mirrored lane holds the other quad's sum. Over 16
// and 32 lanes by swapping register halves with a copy: the two results are the two halves' values in
// all lanes.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v += dpp<kDppXor1>(v);
  if constexpr (L >= 4) v += dpp<kDppXor2>(v);
  if constexpr (L >= 8) v += dpp<kDppMirror8>(v);
  if constexpr (L >= 16) v += dpp<kDppMirror16>(v);
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }
constexpr float kLog2e = 1.44269504088896340736f;
// 1 / (1 + exp(-x)); exp(-x) overflows to infinity, whose reciprocal is 0, for x below about -88.
__device__ __forceinline__ float sigmoid(float x) { return rcp_hw(1.f + exp2_hw(-kLog2e * x)); }

// A launch's threads along one axis stay below 2^32: blocks past 2^20 go to a second axis.
inline dim3 wide_grid(long long blocks) {
  const long long x = blocks < (1 << 20) ? blocks : (1 << 20);
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ long long wide_block() { return (long long)blockIdx.y * gridDim.x + blockIdx.x; }

// Sum of P rows of W fp32 values in a fixed order: thread row ty of kSumRows adds rows ty, ty + kSumRows, ..., eight at
// a time (2^20 rows of equal values: off by 253 times 2^-24, 3327 one by one), then the thread rows are added
// pairwise. out(column, sum) stores it. Few columns per workgroup: a narrow matrix of many rows is spread over more
// CUs, and a thread has a few rounds of loads at most.
constexpr int kSumCols = 16, kSumRows = 64, kSumThreads = kSumCols * kSumRows;
template <class Out>
__device__ __forceinline__ void column_sum_block(const float* __restrict__ part, long long P, int W, int block,
                                                 const Out& out) {
  __shared__ float sm[kSumRows][kSumCols];
  const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
  const int col = block * kSumCols + tx;
  float acc = 0.f;
  if (col < W) {
    const float* p = part + col;
    for (long long r = ty; r < P; r += 8 * kSumRows) {
      float v[8];
      for (int i = 0; i < 8; ++i) {
        const long long k = r + i * kSumRows;
        v[i] = p[(k < P ? k : r) * W];
      }
      float part = 0.f;
      for (int i = 0; i < 8; ++i) part += r + i * kSumRows < P ? v[i] : 0.f;
      acc += part;
    }
  }
  sm[ty][tx] = acc;
  for (int step = kSumRows / 2; step > 0; step /= 2) {
    __syncthreads();
    if (ty < step) sm[ty][tx] += sm[ty + step][tx];
  }
  if (ty == 0 && col < W) out(col, sm[0][tx]);
}
inline int column_sum_blocks(int W) { return (W + kSumCols - 1) / kSumCols; }

template <class Out>
__global__ __launch_bounds__(kSumThreads) void column_sum(const float* __restrict__ part, long long P, int W, Out out) {
  column_sum_block(part, P, W, blockIdx.x, out);
}
template <class Out>
hipError_t column_sum_launch(const float* part, long long P, int W, Out out, hipStream_t st) {
  hipLaunchKernelGGL(column_sum<Out>, dim3((unsigned)column_sum_blocks(W)), dim3(kSumThreads), 0, st, part, P, W, out);
  return hipGetLastError();
}

}  // namespace ttt
