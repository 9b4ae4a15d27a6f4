/*
 * ttt_lm.h -- the operators of a language model's residual block around a TTT layer or a recurrence, in the same
 * library (libttt.so) for AMD Instinct MI355X (gfx950): RMS norm with the residual's addition before it and,
 * for products in 8 bits, a quantised output behind it; dropout; and the gated linear recurrence, a
 * linear-time causal layer with one state per channel. Norm, dropout and recurrence have their
 * backward pass, the recurrence a form for single tokens.
 *
 * Status codes, dtypes, streams, workspaces, errors and threads are ttt.h's; rows, strides, alignment, lengths and
 * precision are ttt_seq.h's. Aliasing: outputs must not overlap any input or each other, except where
 * "in place" is said, and there only as the same rows at the same address.
 *
 * Dropout.  p in [0, 1): each element is zeroed with probability p' = T / 65536, T = p * 65536 rounded to nearest even, and
 *   the others are multiplied by 1 / (1 - p'). p with T = 65536 is refused; with T = 0 nothing is dropped. rng: {seed, offset}, two 64-bit
 *   numbers on the device (8-byte aligned, read when the kernel runs, so that a captured graph draws new masks after
 *   they have been changed there). Element c of row m is dropped where number c % 8 of counter offset + m * ceil(C / 8) + c / 8 is
 *   below T: the eight 16-bit halves, lower first, of the four words of Philox 4x32-10 keyed by the seed at {counter, 0}.
 *   A call uses ttt_dropout_counters(M, C) counters: the next call's offset is that much further on. The backward
 *   pass evaluates them again. Dropped elements are zeros whatever their value.
 */
#ifndef TTT_LM_H_
#define TTT_LM_H_

#include "ttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * RMS norm over each head's D channels. x: M tokens of H heads (token m at x + m * x_stride); weight: fp32 [H, D].
 *   s = x, or residual + dropout(x) where a residual is given,
 *   y = s / sqrt(mean(s^2) + eps) * weight[h].
 * residual, sum, y: [M, H, D]. sum, given exactly when residual is, receives s; it may be the residual in place. The norm is taken
 * of s before it is rounded. A residual needs H = 1, dropout (p > 0, with rng) a residual. D in [1, 16384], H at most
 * 65535, H * D at most 2^24, M * H at most 2^31 - 1; eps finite and not negative. Rows whose sum of squares is past
 * fp32's numbers, above or (with an eps next to zero) below, are normed all the same, as long as they are finite; a row of zeros with an eps of
 * zero is NaN. No workspace.
 */
ttt_status ttt_forward_rmsnorm(ttt_dtype dt, int M, int H, int D, float eps, const void* x, long long x_stride,
                               const void* residual, double p, const long long* rng, const float* weight, void* sum,
                               void* y, void* stream);

/*
 * The same with an output in 8 bits: y: [M, H, D] of e4m3 (4 bits of exponent, 3 of fraction, largest 448, no
 * infinities), scales: fp32 [M, H, D / group]; y * scale is the norm's output,
 *   scale = max |.| of `group` channels / 448 (of 2^-100 where that is larger), y = the nearest to . / scale, ties to even. (The
 * quotient is known to the rounding of s and of the largest to fp32, 2^-24 of it, whatever rows are beside this one.)
 * group: D (one scale for a row), or 32, 64 or 128 where that divides D. A group whose output has a NaN is NaN, scale and all; one whose output
 * has an infinity is NaN there and zeros elsewhere. (Of a row with an infinity in s the norm's output is NaN there and zero elsewhere.)
 */
ttt_status ttt_forward_rmsnorm_e4m3(ttt_dtype dt, int M, int H, int D, int group, float eps, const void* x,
                                    long long x_stride, const void* residual, const float* weight, void* sum, void* y,
                                    float* scales, void* stream);

/*
 * Backward pass. s: what was normed (the forward's x, or sum), token m at s + m * s_stride. With g = d_y * weight, xhat = s / sqrt(..),
 *   d_s = d_sum + (g - xhat * mean(g * xhat)) / sqrt(mean(s^2) + eps),   d_weight[h] = sum_m d_y * xhat,
 *   d_x = d_s with the forward's dropout.
 * d_sum (nullable): the gradient that arrives at sum from elsewhere, [M, H, D]. d_s, the gradient of residual and,
 * without dropout, of x: [M, H, D]; it may be d_sum in place. d_x: [M, D], given exactly when p > 0 (which needs H = 1).
 * d_weight: fp32 [H, D].
 */
ttt_status ttt_backward_rmsnorm(ttt_dtype dt, int M, int H, int D, float eps, const void* s, long long s_stride,
                                const float* weight, const void* d_y, const void* d_sum, double p, const long long* rng,
                                void* d_s, void* d_x, float* d_weight, void* workspace, size_t workspace_bytes,
                                void* stream);
size_t ttt_backward_rmsnorm_workspace(ttt_dtype dt, int M, int H, int D);

/*
 * Dropout of x, M rows of C elements (row m at x + m * x_stride): y = dropout(x), or residual + dropout(x). residual
 * (nullable), y: [M, C]; y may be the residual, or x with a stride of C, in place. The masks are those of ttt_forward_rmsnorm
 * with D = C. C at most 2^24, M * C at most 2^46. rng may be NULL where p is 0.
 */
ttt_status ttt_forward_dropout(ttt_dtype dt, int M, int C, double p, const long long* rng, const void* x,
                               long long x_stride, const void* residual, void* y, void* stream);
/* d_x = dropout(d_y), [M, C] both; d_x may be d_y in place. (A residual's gradient is d_y itself.) */
ttt_status ttt_backward_dropout(ttt_dtype dt, int M, int C, double p, const long long* rng, const void* d_y, void* d_x,
                                void* stream);
long long ttt_dropout_counters(int M, int C);

/*
 * Gated linear recurrence: every channel c keeps a state h,
 *   a = exp(-scale * softplus(lam[c]) * sigmoid(r[b, n, c])),
 *   h = a h + sqrt(1 - a^2) sigmoid(i[b, n, c]) x[b, n, c],   y[b, n, c] = h.
 * x, r, i, y: [B, N, C]; lam: fp32 [C]; h0 (nullable, zeros without it), h_out (nullable): fp32 [B, C], the states before
 * token 0 and after each sequence's last. states (nullable): fp32 [B, ceil(N / 64), C] receives the states before tokens 0, 64,
 * 128, ... (of padding: the sequence's last), which the backward pass can take. scale finite and positive. B at most 65535, N at
 * most 2^22, C at most 2^20, B * (N + 128) * (C + 64) at most 2^38. A NaN, or an infinite x or h0, stays in its channel of its sequence:
 * what is before it is as without it, what is behind it infinite or NaN. Of a state the decays of many tokens may leave nothing (their product is
 * fp32's): what is below 2^-126 of it is lost. Workgroups of a call wait for each other's results; such a wait ends after some seconds
 * whatever happens (a device held up for as long), with TTT_OK, and leaves NaN from its tokens on (backward: up to them).
 */
ttt_status ttt_forward_gated_recurrence(ttt_dtype dt, int B, int N, int C, float scale, const void* x,
                                        long long x_stride, const void* r, long long r_stride, const void* i,
                                        long long i_stride, const float* lam, const float* h0, const int* lengths,
                                        void* y, float* states, float* h_out, void* workspace, size_t workspace_bytes,
                                        void* stream);
size_t ttt_forward_gated_recurrence_workspace(ttt_dtype dt, int B, int N, int C);

/* One token of every sequence: x, r, i, y [B, C] (strides between batch elements); h, h_out: fp32 [B, C], both required; h_out
 * may be h itself. No workspace. */
ttt_status ttt_step_gated_recurrence(ttt_dtype dt, int B, int C, float scale, const void* x, long long x_stride,
                                     const void* r, long long r_stride, const void* i, long long i_stride,
                                     const float* lam, const float* h, void* y, float* h_out, void* stream);

/*
 * Backward pass. With m = sqrt(1 - a^2) and q_n = d_y_n + a_{n+1} q_{n+1} (no gradient flows in through h_out),
 *   d_x = q m sigmoid(i),   d_i = d_x x (1 - sigmoid(i)),
 *   t = q log(a) (a h_{n-1} - (a^2 / m) sigmoid(i) x),   d_r = t (1 - sigmoid(r)),
 *   d_lam = sum_{b, n} t sigmoid(lam) / softplus(lam),   d_h0 = a_0 q_0;
 * log(a) / m is 0 where a is 1. d_y, d_x, d_r, d_i: [B, N, C]; d_lam: fp32 [C]; d_h0 (nullable): fp32 [B, C]. states
 * (nullable): what the forward pass of the same inputs wrote; without them they are computed first.
 */
ttt_status ttt_backward_gated_recurrence(ttt_dtype dt, int B, int N, int C, float scale, const void* x,
                                         long long x_stride, const void* r, long long r_stride, const void* i,
                                         long long i_stride, const float* lam, const float* h0, const int* lengths,
                                         const float* states, const void* d_y, void* d_x, void* d_r, void* d_i,
                                         float* d_lam, float* d_h0, void* workspace, size_t workspace_bytes,
                                         void* stream);
/* `states`: 1 where they will be given, 0 where not. */
size_t ttt_backward_gated_recurrence_workspace(ttt_dtype dt, int B, int N, int C, int states);

#ifdef __cplusplus
}
#endif

#endif /* TTT_LM_H_ */
