"""Binding of the block operators declared in include/ttt_seq.h: layer norm, the short causal convolution and
the selective state space scan, forward, backward and for single tokens.

Argument marshalling only, as in ttt.py, done by the extension module _seq_native (csrc/seq_native.cpp): these
operators take 3 us and up on the device, and a host that marshals with ctypes takes longer than that. Each tensor
is checked against the layout that the C ABI assumes; wrong ones raise TypeError or ValueError, and what the C ABI
itself refuses raises TTTError. Outputs and workspaces that are not passed in are allocated. A call runs on the
current stream of its tensors' device, or on `stream`; buffers it allocates belong to that stream.

As with the layers of ttt.py, autograd has no part in a call: outputs carry no gradient function (nor a forward-mode
tangent) even where an input requires gradients; a torch.autograd.Function made of a forward and a backward call gives
them one. Tensors that a call writes, states in place among them, count as changed in place, so that autograd refuses
gradients that need their old values.
"""
from __future__ import annotations

import os

from .ttt import _raise, _torch, load_library

_module = None


def _native():
    """The extension module, bound to the loaded libttt.so; raises if either has not been built."""
    global _module
    if _module is None:
        _torch()  # (the module's symbols come from PyTorch's libraries)
        handle = load_library()._handle
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_seq_native.so")
        if not os.path.exists(path):
            raise RuntimeError(f"_seq_native.so not built ({path}); run __graft_entry__.build() or "
                               "python -m test_sequence_layers_amd.build")
        from . import _seq_native
        _seq_native.bind(handle)
        _module = _seq_native
    return _module


def _call(where, stream, fn, *args):
    """fn's outputs; a status that it returns in their place raises TTTError."""
    if stream is None:
        r = fn(*args)
    else:
        torch = _torch()
        x = args[0]
        if isinstance(x, torch.Tensor) and x.is_cuda and x.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, not {x.device}")
        with torch.cuda.stream(stream):
            r = fn(*args)
    if type(r) is int:
        _raise(r, where)
    return r


# ---------------------------------------------------------------------------------- layer norm
def ttt_forward_layernorm(x, weight, bias=None, eps: float = 1e-5, *, y=None, stream=None):
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dim. Returns y (x's shape).

    x: [..., D] with weight, bias fp32 [D], or [..., H, D] with [H, D] (each head normed by its own row);
    bf16 or fp32; x may be a slice whose rows are evenly spaced."""
    return _call("ttt_forward_layernorm", stream, _native().layernorm_forward, x, weight, bias, eps, y)


def ttt_backward_layernorm(x, weight, d_y, eps: float = 1e-5, *, d_x=None, d_weight=None, d_bias=None, workspace=None,
                           stream=None):
    """Gradients (d_x, d_weight, d_bias) of ttt_forward_layernorm given d_y (contiguous, x's shape)."""
    return _call("ttt_backward_layernorm", stream, _native().layernorm_backward,
                 x, weight, d_y, eps, d_x, d_weight, d_bias, workspace)


# ------------------------------------------------------------------- short causal convolution
def ttt_forward_conv1d(x, weight, bias=None, *, silu: bool = False, state=None, lengths=None, state_out=None, y=None,
                       stream=None):
    """Causal depth-wise convolution over the tokens: bias[c] + sum_k weight[c, k] x[b, n - (K - 1) + k, c],
    then SiLU if asked. Returns y [B, N, C].

    x: [B, N, C] bf16 or fp32 (a slice of wider rows is read in place); weight fp32 [C, K], K = 2..4; bias fp32
    [C]; state: [B, K - 1, C] of x's dtype, the inputs before token 0 (zeros without it); lengths: int32 [B],
    the tokens of each sequence (y is zero behind them); state_out: receives the last K - 1 inputs."""
    return _call("ttt_forward_conv1d", stream, _native().conv1d_forward,
                 x, weight, bias, silu, state, lengths, state_out, y)


def ttt_step_conv1d(x, weight, bias=None, *, state, silu: bool = False, state_out=None, y=None, stream=None):
    """One token of every sequence: x [B, C], state [B, K - 1, C] its last inputs, updated in place unless
    state_out is given. Returns y [B, C]."""
    return _call("ttt_step_conv1d", stream, _native().conv1d_step, x, weight, bias, silu, state, state_out, y)


def ttt_backward_conv1d(x, weight, bias, d_y, *, silu: bool = False, state=None, lengths=None, d_x=None, d_weight=None,
                        d_bias=None, d_state=None, workspace=None, stream=None):
    """Gradients (d_x, d_weight, d_bias, d_state) of ttt_forward_conv1d given d_y (contiguous [B, N, C]); no
    gradient flows in through state_out. d_state is None without a state, d_bias without a bias."""
    return _call("ttt_backward_conv1d", stream, _native().conv1d_backward,
                 x, weight, bias, d_y, silu, state, lengths, d_x, d_weight, d_bias, d_state, workspace)


# ---------------------------------------------------------------------- selective state space scan
def ttt_forward_selective_scan(u, delta, A, Bm, Cm, D=None, delta_bias=None, z=None, *, softplus: bool = True, h0=None,
                               lengths=None, h_out=None, y=None, workspace=None, stream=None):
    """h = exp(step A) h + step Bm u, y = (Cm . h + D u) * SiLU(z), step = softplus(delta + delta_bias), per channel
    and token. Returns y [B, N, C].

    u, delta, z: [B, N, C] bf16 or fp32; Bm, Cm: [B, N, G, S] (slices of wider rows are read in place); A fp32
    [C, S], S in {8, 16, 32, 64}; D, delta_bias fp32 [C]; h0, h_out: fp32 [B, C, S], the states before the first and
    after the last token; lengths: int32 [B], the tokens of each sequence (y is zero behind them)."""
    return _call("ttt_forward_selective_scan", stream, _native().scan_forward,
                 u, delta, A, Bm, Cm, D, delta_bias, z, softplus, h0, lengths, h_out, y, workspace)


def ttt_step_selective_scan(u, delta, A, Bm, Cm, D=None, delta_bias=None, z=None, *, h, softplus: bool = True, h_out=None,
                            y=None, stream=None):
    """One token of every sequence: u, delta, z [B, C], Bm, Cm [B, G, S]; h fp32 [B, C, S], updated in place unless
    h_out is given. Returns y [B, C]."""
    return _call("ttt_step_selective_scan", stream, _native().scan_step,
                 u, delta, A, Bm, Cm, D, delta_bias, z, softplus, h, h_out, y)


def ttt_backward_selective_scan(u, delta, A, Bm, Cm, d_y, D=None, delta_bias=None, z=None, *, softplus: bool = True,
                                h0=None, lengths=None, d_u=None, d_delta=None, d_A=None, d_B=None, d_C=None, d_D=None,
                                d_delta_bias=None, d_z=None, d_h0=None, workspace=None, stream=None):
    """Gradients (d_u, d_delta, d_A, d_B, d_C, d_D, d_delta_bias, d_z, d_h0) of ttt_forward_selective_scan given d_y
    (contiguous [B, N, C]); those of inputs that are None are None. No gradient flows in through h_out."""
    return _call("ttt_backward_selective_scan", stream, _native().scan_backward,
                 u, delta, A, Bm, Cm, D, delta_bias, z, softplus,
                 h0, lengths, d_y, d_u, d_delta, d_A, d_B, d_C, d_D, d_delta_bias, d_z, d_h0, workspace)
