// Host-side interface between the C ABI of the block operators (abi_seq.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace ttt {

// ---- layer norm -------------------------------------------------------------------------------
hipError_t layernorm_launch(bool bf16_io, int M, int H, int D, float eps, const void* x, long long xs,
                            const float* w, const float* b, void* y, hipStream_t st);
size_t layernorm_bwd_workspace_bytes(bool bf16_io, int M, int H, int D);
hipError_t layernorm_bwd_launch(bool bf16_io, int M, int H, int D, float eps, const void* x,
                                long long xs, const float* w, const void* dy, void* dx, float* dw,
                                float* db, void* ws, hipStream_t st);

// ---- short causal convolution -----------------------------------------------------------------
struct Conv1dArgs {
  int B, N, C;
  const void* x;
  long long xs;  // elements between tokens
  const float* w;
  const float* bias;
  const void* state;
  const int* lengths;
  void* y;          // forward, step
  void* state_out;  // forward, step
  const void* dy;   // backward, from here on
  void* dx;
  float* dw;
  float* db;
  void* dstate;
  float* partial;
};
hipError_t conv1d_launch(bool bf16_io, int K, bool silu, const Conv1dArgs& a, hipStream_t st);
hipError_t conv1d_step_launch(bool bf16_io, int K, bool silu, const Conv1dArgs& a, hipStream_t st);
size_t conv1d_bwd_workspace_bytes(bool bf16_io, int B, int N, int C, int K);
hipError_t conv1d_bwd_launch(bool bf16_io, int K, bool silu, const Conv1dArgs& a, hipStream_t st);

// ---- selective state space scan ---------------------------------------------------------------
struct ScanArgs {
  int B, N, C, G;
  int softplus;
  const void *u, *delta, *bm, *cm, *z;
  long long us, ds, bs, cs, zs;  // elements between tokens
  const float *A, *D, *dbias, *h0;
  const int* lengths;
  void* y;
  float* h_out;
  const void* dy;  // backward, from here on
  void *du, *ddelta, *dbm, *dcm, *dz;
  float *dA, *dD, *ddbias, *dh0;
};
bool scan_supported_s(int S);
size_t scan_workspace_bytes(bool bf16_io, int B, int N, int C, int S, int G);
hipError_t scan_launch(bool bf16_io, int S, const ScanArgs& a, void* ws, hipStream_t st);
hipError_t scan_step_launch(bool bf16_io, int S, const ScanArgs& a, hipStream_t st);
size_t scan_bwd_workspace_bytes(bool bf16_io, int B, int N, int C, int S, int G);
hipError_t scan_bwd_launch(bool bf16_io, int S, const ScanArgs& a, void* ws, hipStream_t st);

}  // namespace ttt
