/*
 * ttt_seq.h -- the operators of a sequence block around and beside a TTT layer, in the same library
 * (libttt.so) for AMD Instinct MI355X (gfx950): layer norm (a block is Norm -> layer -> residual,
 * ViT^3 review on techloop.online, "TTT Block" section; a TTT layer also norms each head's queries
 * and keys), the short causal convolution before a causal layer, and the selective state space
 * scan, the other linear-time causal layer. Each has its forward and backward pass, and the two
 * causal ones a form for single tokens.
 *
 * Status codes, dtypes, streams, workspaces, errors and threads are ttt.h's, with these differences:
 *
 * Rows.  Activations are [B, N, C] (or [M, H, D]) with the channels contiguous. Where an argument is
 *   followed by a stride, token n of batch b starts `stride` elements after the token before it
 *   (token b * N + n at that multiple), so that a slice of a wider projection's rows is read in
 *   place; a stride is at least the row's width. Everything else is contiguous.
 * Alignment.  Pointers need the alignment of their elements. Where every pointer and row is 16-byte
 *   aligned (x, y, d_y, d_x and the weights), the 16-byte paths run; results are the same up to
 *   rounding either way.
 * Lengths.  `lengths` (nullable): int32 [B] on the device, sequence b's number of tokens, in [0, N]
 *   (values outside are taken as the nearer end). The tokens behind it are padding: nothing
 *   depends on their values, states pass over them, and their rows of y and of every gradient are written as zeros.
 * Aliasing.  Outputs must not overlap any input or each other, except that a step's state may be
 *   updated in place.
 * Precision.  Everything is computed and summed in fp32 and rounded once, to nearest even, on
 *   output. Sums are in a fixed order: the same call gives the same bits.
 */
#ifndef TTT_SEQ_H_
#define TTT_SEQ_H_

#include "ttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm over each head's D channels. x: M tokens of H heads (token m at x + m * x_stride, its
 * heads' D channels back to back); weight, bias (nullable): fp32 [H, D]; y: [M, H, D].
 *   y = (x - mean) / sqrt(var + eps) * weight[h] + bias[h],
 * mean and var (the population variance, from the centred values) over the D channels. H = 1 is the
 * ordinary layer norm of a row; H > 1 with D the head width norms queries or keys per head.
 * D in [1, 16384], H at most 65535, H * D at most 2^24, M * H at most 2^31 - 1; eps finite and not
 * negative. No workspace.
 */
ttt_status ttt_forward_layernorm(ttt_dtype dt, int M, int H, int D, float eps, const void* x,
                                 long long x_stride, const float* weight, const float* bias,
                                 void* y, void* stream);

/*
 * Backward pass: with g = d_y * weight and xhat the normed x (recomputed from x),
 *   d_x = (g - mean(g) - xhat * mean(g * xhat)) / sqrt(var + eps),
 *   d_weight[h] = sum_m d_y * xhat,   d_bias[h] = sum_m d_y.
 * d_y, d_x: [M, H, D]; d_weight, d_bias (nullable): fp32 [H, D].
 */
ttt_status ttt_backward_layernorm(ttt_dtype dt, int M, int H, int D, float eps, const void* x,
                                  long long x_stride, const float* weight, const void* d_y,
                                  void* d_x, float* d_weight, float* d_bias, void* workspace,
                                  size_t workspace_bytes, void* stream);
size_t ttt_backward_layernorm_workspace(ttt_dtype dt, int M, int H, int D);

/*
 * Short causal depth-wise convolution: K taps per channel over the token and the K - 1 before it,
 *   pre[b, n, c] = bias[c] + sum_{k = 0..K-1} weight[c, k] x[b, n - (K - 1) + k, c],
 *   y = pre, or pre * sigmoid(pre) when silu is 1.
 * weight: fp32 [C, K]; bias: fp32 [C] or NULL; y: [B, N, C]. state (nullable): [B, K - 1, C] of dtype
 * dt, the inputs before token 0 (zeros without it); state_out (nullable): [B, K - 1, C] receives the
 * last K - 1 inputs of each sequence (the state's own where it is shorter), so that a later call
 * continues it. K in {2, 3, 4}; B at most 65535, N at most 2^22, C at most 2^20. No workspace.
 */
ttt_status ttt_forward_conv1d(ttt_dtype dt, int B, int N, int C, int K, int silu, const void* x,
                              long long x_stride, const float* weight, const float* bias,
                              const void* state, const int* lengths, void* y, void* state_out,
                              void* stream);

/* One token of every sequence: x [B, C] (token b at x + b * x_stride), y [B, C]; state and state_out as
 * above, both required; state_out may be state itself. */
ttt_status ttt_step_conv1d(ttt_dtype dt, int B, int C, int K, int silu, const void* x,
                           long long x_stride, const float* weight, const float* bias,
                           const void* state, void* y, void* state_out, void* stream);

/*
 * Backward pass: with d_pre = d_y * act'(pre) (pre recomputed from x), zero outside the sequence,
 *   d_x[n] = sum_k weight[k] d_pre[n + K - 1 - k],   d_weight[k] = sum_{b, n} d_pre[n] x[n - (K - 1) + k],
 *   d_bias = sum_{b, n} d_pre.
 * d_y, d_x: [B, N, C]; d_weight: fp32 [C, K]; d_bias (nullable): fp32 [C]; d_state (nullable, only
 * with a state): [B, K - 1, C] of dtype dt, the gradient of the inputs before token 0.
 */
ttt_status ttt_backward_conv1d(ttt_dtype dt, int B, int N, int C, int K, int silu, const void* x,
                               long long x_stride, const float* weight, const float* bias,
                               const void* state, const int* lengths, const void* d_y, void* d_x,
                               float* d_weight, float* d_bias, void* d_state, void* workspace,
                               size_t workspace_bytes, void* stream);
size_t ttt_backward_conv1d_workspace(ttt_dtype dt, int B, int N, int C, int K);

/*
 * Selective state space scan: every channel c keeps a state h of S numbers,
 *   step = softplus(delta[b, n, c] + delta_bias[c])   (the sum itself when softplus is 0),
 *   h[s] = exp(step * A[c, s]) h[s] + step * Bm[b, n, g, s] * u[b, n, c],
 *   y[b, n, c] = (sum_s Cm[b, n, g, s] h[s] + D[c] u[b, n, c]) * (z sigmoid(z) when z is given),
 * g = c / (C / G). u, delta, z (nullable), y: [B, N, C]; Bm, Cm: [B, N, G, S]; A: fp32 [C, S]; D,
 * delta_bias (nullable): fp32 [C]; h0 (nullable, zeros without it), h_out (nullable): fp32 [B, C, S],
 * the states before token 0 and after each sequence's last. S in {8, 16, 32, 64}; G divides C; B at
 * most 65535, N at most 2^22, C at most 2^20, B * C * (N + 4096) at most 2^38, B * G *
 * ceil(C / G / 64) at most 2^20. For bf16, Bm and Cm are 4-byte aligned and their strides even, in every
 * form. Tokens are taken in segments at once, from the states that products of decays give: where step * A is
 * positive and exp of its sum over some tokens is not finite in fp32, states other than zero are not either.
 */
ttt_status ttt_forward_selective_scan(ttt_dtype dt, int B, int N, int C, int S, int G, int softplus,
                                      const void* u, long long u_stride, const void* delta,
                                      long long delta_stride, const float* A, const void* Bm,
                                      long long b_stride, const void* Cm, long long c_stride,
                                      const float* D, const float* delta_bias, const void* z,
                                      long long z_stride, const float* h0, const int* lengths,
                                      void* y, float* h_out, void* workspace,
                                      size_t workspace_bytes, void* stream);
size_t ttt_forward_selective_scan_workspace(ttt_dtype dt, int B, int N, int C, int S, int G);

/* One token of every sequence: u, delta, z, y [B, C], Bm, Cm [B, G, S] (strides between batch elements);
 * h, h_out: fp32 [B, C, S], both required; h_out may be h itself. No workspace. */
ttt_status ttt_step_selective_scan(ttt_dtype dt, int B, int C, int S, int G, int softplus,
                                   const void* u, long long u_stride, const void* delta,
                                   long long delta_stride, const float* A, const void* Bm,
                                   long long b_stride, const void* Cm, long long c_stride,
                                   const float* D, const float* delta_bias, const void* z,
                                   long long z_stride, const float* h, void* y, float* h_out,
                                   void* stream);

/*
 * Backward pass. With a_n = exp(step_n A), v = d_y * (z sigmoid(z)), and
 *   q_n = v_n Cm_n + a_{n+1} q_{n+1}   (the gradient of the state after token n; no gradient flows in
 *                                      through h_out),
 *   d_u = step * sum_s q Bm + D v,
 *   d_step = sum_s q (A a h_{n-1} + Bm u),   d_delta = d_step * softplus'(delta + delta_bias),
 *   d_A = sum_{b, n} q a h_{n-1} step,   d_B = sum_{c in g} q step u,   d_C = sum_{c in g} v h_n,
 *   d_D = sum_{b, n} v u,   d_delta_bias = sum_{b, n} d_delta,   d_h0 = a_0 q_0,
 *   d_z = d_y (sum_s Cm h + D u) (z sigmoid(z))'.
 * d_u, d_delta, d_z: [B, N, C]; d_B, d_C: [B, N, G, S] of dtype dt; d_A: fp32 [C, S]; d_D, d_delta_bias:
 * fp32 [C]; d_h0: fp32 [B, C, S]. d_z is given exactly when z is; d_D, d_delta_bias and d_h0 may be
 * NULL. The forward pass is recomputed from the inputs, nothing of it has to be kept. step * A must not be
 * positive by so much that exp of its sum over a run of tokens is infinite in fp32: gradients are NaN then, also
 * where states or d_y are zeros.
 * The workspace holds states every 8 tokens and each block of 64 channels' sums for d_B and d_C: about 5 S / 8 + 1 bytes per
 * token and channel where a group's channels are whole blocks (the sums are 8 S bytes per token and block), and 12 (S + 1)
 * per channel and segment of 16 to 2048 tokens: 106 MB for bf16 2 x 4096 x 768 x 16, 5.5 GB for 8 x 8192 x 2048 x 64.
 */
ttt_status ttt_backward_selective_scan(ttt_dtype dt, int B, int N, int C, int S, int G, int softplus,
                                       const void* u, long long u_stride, const void* delta,
                                       long long delta_stride, const float* A, const void* Bm,
                                       long long b_stride, const void* Cm, long long c_stride,
                                       const float* D, const float* delta_bias, const void* z,
                                       long long z_stride, const float* h0, const int* lengths,
                                       const void* d_y, void* d_u, void* d_delta, float* d_A,
                                       void* d_B, void* d_C, float* d_D, float* d_delta_bias,
                                       void* d_z, float* d_h0, void* workspace,
                                       size_t workspace_bytes, void* stream);
size_t ttt_backward_selective_scan_workspace(ttt_dtype dt, int B, int N, int C, int S, int G);

#ifdef __cplusplus
}
#endif

#endif /* TTT_SEQ_H_ */
