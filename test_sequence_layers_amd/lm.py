"""Binding of the residual block's operators declared in include/ttt_lm.h: RMS norm with the residual's addition and an
output in 8 bits, dropout, and the gated linear recurrence, forward, backward and for single tokens.

As seq.py's: argument marshalling only, by the same extension module (csrc/lm_native.cpp); tensors are checked against the
layout that the C ABI assumes (TypeError, ValueError), what the C ABI refuses raises TTTError, outputs and workspaces that are not
passed in are allocated, a call runs on the current stream or on `stream`, autograd has no part in it, and tensors
that it writes count as changed in place.

Dropout's random numbers are a function of rng, an int64 tensor (seed, offset) on the device, and of an element's place: the
same rng gives the same mask, forward and backward. A call uses dropout_counters(x) of its counters; add them to the offset (on
the device, also inside a captured graph) before the next mask is drawn.
"""
from __future__ import annotations

from .seq import _call, _native
from .ttt import load_library


# ----------------------------------------------------------------------------------- RMS norm
def ttt_forward_rmsnorm(x, weight, eps: float = 1e-5, *, residual=None, p: float = 0.0, rng=None, sum_out=None, y=None,
                        stream=None):
    """s / sqrt(mean(s^2) + eps) * weight over the last dim, s = x or residual + dropout(x, p). Returns y (x's shape), with
    a residual (y, sum), sum being s.

    x: [..., D] with weight fp32 [D], or [..., H, D] with [H, D] (each head normed by its own row; without a residual); bf16 or
    fp32; x may be a slice whose rows are evenly spaced; residual: contiguous, x's shape; sum_out may be the residual (in place)."""
    return _call("ttt_forward_rmsnorm", stream, _native().rmsnorm_forward, x, weight, eps, residual, p, rng, sum_out, y)


def ttt_forward_rmsnorm_e4m3(x, weight, eps: float = 1e-5, *, residual=None, group: int = 0, sum_out=None, y=None,
                             scales=None, stream=None):
    """The same (without dropout) in 8 bits: returns (y, scales), with a residual (y, scales, sum). y: float8_e4m3fn of x's shape;
    scales: fp32 [..., D / group], the largest of each `group` channels / 448; y * scales is the norm's output. group: 0 (the
    whole row), 32, 64 or 128."""
    return _call("ttt_forward_rmsnorm_e4m3", stream, _native().rmsnorm_e4m3, x, weight, eps, residual, group, sum_out, y,
                 scales)


def ttt_backward_rmsnorm(s, weight, d_y, eps: float = 1e-5, *, d_sum=None, p: float = 0.0, rng=None, d_s=None, d_x=None,
                         d_weight=None, workspace=None, stream=None):
    """Gradients (d_s, d_x, d_weight) given d_y and, where sum is used elsewhere too, its gradient d_sum from there (contiguous,
    s's shape). s: what was normed, the forward's x or its sum. d_s is the gradient of residual and, without dropout, of x; d_x
    is None then, and x's gradient through the dropout where p is not 0. d_s may be d_sum (in place)."""
    return _call("ttt_backward_rmsnorm", stream, _native().rmsnorm_backward,
                 s, weight, d_y, eps, d_sum, p, rng, d_s, d_x, d_weight, workspace)


# ----------------------------------------------------------------------------------- dropout
def ttt_forward_dropout(x, p: float, rng, *, residual=None, y=None, stream=None):
    """x with each element zeroed with probability p and the others divided by 1 - p, added to the residual if there is one.
    Returns y (x's shape), which may be given as x or residual themselves. p is taken to the nearest 65536th."""
    return _call("ttt_forward_dropout", stream, _native().dropout_forward, x, p, rng, residual, y)


def ttt_backward_dropout(d_y, p: float, rng, *, d_x=None, stream=None):
    """x's gradient: d_y (contiguous) with the mask of the forward call. d_x may be d_y itself."""
    return _call("ttt_backward_dropout", stream, _native().dropout_backward, d_y, p, rng, d_x)


def dropout_counters(x) -> int:
    """How many counters one mask of x's shape uses: what to add to rng's offset before the next."""
    C = x.shape[-1]
    return int(load_library().ttt_dropout_counters(x.numel() // C if C else 0, C))


# ----------------------------------------------------------------------- gated linear recurrence
def ttt_forward_gated_recurrence(x, r, i, lam, *, scale: float = 8.0, h0=None, lengths=None, states=None, h_out=None, y=None,
                                 workspace=None, stream=None):
    """h = a h + sqrt(1 - a^2) sigmoid(i) x, a = exp(-scale softplus(lam) sigmoid(r)), per channel and token. Returns y = h,
    [B, N, C].

    x, r, i: [B, N, C] bf16 or fp32 (slices of wider rows are read in place); lam fp32 [C]; h0, h_out: fp32 [B, C], the states
    before the first and after the last token; lengths: int32 [B], the tokens of each sequence (y is zero behind them);
    states: fp32 [B, ceil(N / 64), C], receives the state before every 64th token, for the backward pass."""
    return _call("ttt_forward_gated_recurrence", stream, _native().recurrence_forward,
                 x, r, i, lam, scale, h0, lengths, states, h_out, y, workspace)


def ttt_step_gated_recurrence(x, r, i, lam, *, h, scale: float = 8.0, h_out=None, y=None, stream=None):
    """One token of every sequence: x, r, i [B, C]; h fp32 [B, C], updated in place unless h_out is given. Returns y [B, C]."""
    return _call("ttt_step_gated_recurrence", stream, _native().recurrence_step, x, r, i, lam, scale, h, h_out, y)


def ttt_backward_gated_recurrence(x, r, i, lam, d_y, *, scale: float = 8.0, h0=None, lengths=None, states=None, d_x=None,
                                  d_r=None, d_i=None, d_lam=None, d_h0=None, workspace=None, stream=None):
    """Gradients (d_x, d_r, d_i, d_lam, d_h0) of ttt_forward_gated_recurrence given d_y (contiguous [B, N, C]); d_h0 is None
    without h0. states: what the forward call on the same inputs wrote; without them they are computed first. No
    gradient flows in through h_out."""
    return _call("ttt_backward_gated_recurrence", stream, _native().recurrence_backward,
                 x, r, i, lam, scale, h0, lengths, states, d_y, d_x, d_r, d_i, d_lam, d_h0, workspace)
