// Host-side interface between the C ABI of ttt_lm.h (abi_lm.hip) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "philox.hpp"

namespace ttt {

// ---- RMS norm ---------------------------------------------------------------------------------
struct RmsNormArgs {
  int M, H, D, group;
  float eps;
  const void* x;   // forward: what is added or normed; backward: what was normed
  long long xs;    // elements between tokens
  const float* w;
  Drop drop;
  const void* residual;  // forward
  void *sum, *y;
  float* scales;
  const void *dy, *dsum;  // backward
  void *ds, *dx;
  float *dw, *partial;
};
hipError_t rmsnorm_launch(bool bf16_io, const RmsNormArgs& a, hipStream_t st);
size_t rmsnorm_bwd_workspace_bytes(bool bf16_io, int M, int H, int D);
hipError_t rmsnorm_bwd_launch(bool bf16_io, const RmsNormArgs& a, hipStream_t st);

// ---- dropout ----------------------------------------------------------------------------------
struct DropoutArgs {
  int M, C;
  const void* x;
  long long xs;
  const void* residual;
  void* y;
  Drop drop;
};
hipError_t dropout_launch(bool bf16_io, const DropoutArgs& a, hipStream_t st);

// ---- gated recurrence -------------------------------------------------------------------------
constexpr int kKept = 64;  // tokens between the recurrence's kept states
struct RecurrenceArgs {
  int B, N, C;
  float scale;
  const void *x, *r, *i;
  long long xs, rs, is;  // elements between tokens
  const float *lam, *h0;
  const int* lengths;
  void* y;                  // forward, step
  float *states, *h_out;    // forward, step
  const float* kept;        // backward: the forward pass's states
  const void* dy;           // backward, from here on
  void *dx, *dr, *di;
  float *dlam, *dh0;
};
size_t recurrence_workspace_bytes(bool bf16_io, int B, int N, int C);
hipError_t recurrence_launch(bool bf16_io, const RecurrenceArgs& a, void* ws, hipStream_t st);
hipError_t recurrence_step_launch(bool bf16_io, const RecurrenceArgs& a, hipStream_t st);
size_t recurrence_bwd_workspace_bytes(bool bf16_io, int B, int N, int C, bool kept);
hipError_t recurrence_bwd_launch(bool bf16_io, const RecurrenceArgs& a, void* ws, hipStream_t st);

}  // namespace ttt
