"""ctypes binding of the block operators declared in include/ttt_seq.h: layer norm, the short causal
convolution and the selective state space scan, forward, backward and for single tokens.

Argument marshalling only, as in ttt.py: the binding sees the tensors' shapes and checks each against
the layout the C ABI assumes. Buffers it allocates itself (outputs and workspaces not passed in)
belong to the stream that the call runs on.
"""
from __future__ import annotations

from .ttt import _dtype_code, _raise, _torch, load_library

torch = None  # bound by the first call: the package itself loads without torch


class _Call:
    """The device, dtype and stream of one call, and the checks of its tensors against them.

    A single-token call takes a few microseconds on the device, so the checks cost as little host time as
    they can: each tensor is compared with what it should be at once, and only one that differs is
    looked at piece by piece for the error's text."""

    def __init__(self, name, x, stream):
        global torch
        if torch is None:
            torch = _torch()
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        self.device, self.io = x.device, x.dtype
        self.dt = _dtype_code(x)
        self.stream = stream

    def _refuse(self, name, t, dtype, shape):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, not {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must have dtype {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")

    def need(self, name, t, shape, dtype=None):
        """Data pointer of a contiguous tensor, fp32 unless told otherwise."""
        if dtype is None:
            dtype = torch.float32
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == self.device
                and t.is_contiguous()):
            return t.data_ptr()
        self._refuse(name, t, dtype, shape)

    def dense(self, name, t, shape, dtype=None):
        """The same of a tensor that may be left out; None for None."""
        return None if t is None else self.need(name, t, shape, dtype)

    def rows(self, name, t, shape, width):
        """(data pointer, elements between rows) of an activation whose last dims (`width` elements) are
        contiguous and whose leading dims are one run of evenly spaced rows."""
        if not (isinstance(t, torch.Tensor) and t.dtype is self.io and t.shape == shape and t.device == self.device):
            self._refuse(name, t, self.io, shape)
        if t.is_contiguous():
            return t.data_ptr(), width
        sizes, strides = t.shape, t.stride()
        inner, d = 1, len(sizes)
        while inner < width:  # the dims that make up a row
            d -= 1
            if sizes[d] != 1 and strides[d] != inner:
                raise ValueError(f"the last {width} elements of each row of {name} must be contiguous")
            inner *= sizes[d]
        step = span = None
        for i in range(d - 1, -1, -1):
            if sizes[i] == 1:
                continue
            if step is None:
                step = strides[i]
            elif strides[i] != span:
                raise ValueError(f"the rows of {name} must be evenly spaced over its leading dims")
            span = strides[i] * sizes[i]
        step = width if step is None else step
        if step < width:
            raise ValueError(f"the rows of {name} overlap")
        return t.data_ptr(), step

    def empty(self, shape, dtype):
        if self.stream is not None:
            with torch.cuda.stream(self.stream):
                return torch.empty(shape, dtype=dtype, device=self.device)
        return torch.empty(shape, dtype=dtype, device=self.device)

    def output(self, name, t, like):
        """(tensor, pointer) of an output of `like`'s shape and dtype, allocated if it was not passed in."""
        if t is not None:
            return t, self.need(name, t, like.shape, like.dtype)
        if self.stream is None:  # (empty_like takes half the host time of empty)
            t = torch.empty_like(like, memory_format=torch.contiguous_format)
        else:
            t = self.empty(like.shape, like.dtype)
        return t, t.data_ptr()

    def workspace(self, t, need):
        """(tensor, pointer, bytes)."""
        if t is None:
            if need == 0:
                return None, None, 0
            t = self.empty((need,), torch.uint8)
        elif not isinstance(t, torch.Tensor) or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        return t, t.data_ptr(), t.numel() * t.element_size()

    def lengths(self, t, B):
        return None if t is None else self.need("lengths", t, (B,), torch.int32)

    def run(self, fn_name, *args):
        fn = getattr(load_library(), fn_name)
        index = self.device.index
        # (the handle itself: torch.cuda.current_stream makes an object first, a tenth of a small call)
        s = torch._C._cuda_getCurrentRawStream(index) if self.stream is None else self.stream.cuda_stream
        if index == torch.cuda.current_device():
            st = fn(*args, s)
        else:
            with torch.cuda.device(index):
                st = fn(*args, s)
        if st:
            _raise(st, fn_name)


# ---------------------------------------------------------------------------------- layer norm
def _norm_shape(x, weight):
    """(M, H, D): weight [D] norms x's rows, weight [H, D] each head's D of [..., H, D]."""
    shape = weight.shape if isinstance(weight, torch.Tensor) else ()
    nd = len(shape)
    if nd not in (1, 2):
        raise ValueError("weight must be [D] or [H, D]")
    if x.dim() <= nd or x.shape[-nd:] != shape:
        raise ValueError(f"x must be [..., {', '.join(map(str, shape))}], not {tuple(x.shape)}")
    H, D = (1, shape[0]) if nd == 1 else shape
    return x.numel() // max(H * D, 1), H, D


def ttt_forward_layernorm(x, weight, bias=None, eps: float = 1e-5, *, y=None, stream=None):
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dim. Returns y (x's shape).

    x: [..., D] with weight, bias fp32 [D], or [..., H, D] with [H, D] (each head normed by its own row);
    bf16 or fp32; x may be a slice whose rows are evenly spaced."""
    call = _Call("x", x, stream)
    M, H, D = _norm_shape(x, weight)
    px, xs = call.rows("x", x, x.shape, H * D)
    pw, pb = call.need("weight", weight, weight.shape), call.dense("bias", bias, weight.shape)
    y, py = call.output("y", y, x)
    call.run("ttt_forward_layernorm", call.dt, M, H, D, float(eps), px, xs, pw, pb, py)
    return y


def ttt_backward_layernorm(x, weight, d_y, eps: float = 1e-5, *, d_x=None, d_weight=None, d_bias=None, workspace=None,
                           stream=None):
    """Gradients (d_x, d_weight, d_bias) of ttt_forward_layernorm given d_y (contiguous, x's shape)."""
    call = _Call("x", x, stream)
    M, H, D = _norm_shape(x, weight)
    px, xs = call.rows("x", x, x.shape, H * D)
    pw, pdy = call.need("weight", weight, weight.shape), call.need("d_y", d_y, x.shape, call.io)
    d_x, pdx = call.output("d_x", d_x, x)
    d_weight, pdw = call.output("d_weight", d_weight, weight)
    d_bias, pdb = call.output("d_bias", d_bias, weight)
    workspace, pws, nws = call.workspace(workspace, load_library().ttt_backward_layernorm_workspace(call.dt, M, H, D))
    call.run("ttt_backward_layernorm", call.dt, M, H, D, float(eps), px, xs, pw, pdy, pdx, pdw, pdb, pws, nws)
    return d_x, d_weight, d_bias


# ------------------------------------------------------------------- short causal convolution
def _conv_shape(x, weight, dims):
    if x.dim() != dims:
        raise ValueError("x must be [B, N, C]" if dims == 3 else "x must be [B, C]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, K]")
    return x.shape[0], x.shape[1] if dims == 3 else 1, x.shape[-1], weight.shape[1]


def ttt_forward_conv1d(x, weight, bias=None, *, silu: bool = False, state=None, lengths=None, state_out=None, y=None,
                       stream=None):
    """Causal depth-wise convolution over the tokens: bias[c] + sum_k weight[c, k] x[b, n - (K - 1) + k, c],
    then SiLU if asked. Returns y [B, N, C].

    x: [B, N, C] bf16 or fp32 (a slice of wider rows is read in place); weight fp32 [C, K], K = 2..4; bias fp32
    [C]; state: [B, K - 1, C] of x's dtype, the inputs before token 0 (zeros without it); lengths: int32 [B],
    the tokens of each sequence (y is zero behind them); state_out: receives the last K - 1 inputs."""
    call = _Call("x", x, stream)
    B, N, C, K = _conv_shape(x, weight, 3)
    px, xs = call.rows("x", x, x.shape, C)
    pw, pb = call.need("weight", weight, (C, K)), call.dense("bias", bias, (C,))
    held = (B, K - 1, C)
    ps, pl = call.dense("state", state, held, call.io), call.lengths(lengths, B)
    pso = call.dense("state_out", state_out, held, call.io)
    y, py = call.output("y", y, x)
    call.run("ttt_forward_conv1d", call.dt, B, N, C, K, int(bool(silu)), px, xs, pw, pb, ps, pl, py, pso)
    return y


def ttt_step_conv1d(x, weight, bias=None, *, state, silu: bool = False, state_out=None, y=None, stream=None):
    """One token of every sequence: x [B, C], state [B, K - 1, C] its last inputs, updated in place unless
    state_out is given. Returns y [B, C]."""
    call = _Call("x", x, stream)
    B, _, C, K = _conv_shape(x, weight, 2)
    px, xs = call.rows("x", x, x.shape, C)
    pw, pb = call.need("weight", weight, (C, K)), call.dense("bias", bias, (C,))
    ps = call.need("state", state, (B, K - 1, C), call.io)
    pso = ps if state_out is None else call.dense("state_out", state_out, (B, K - 1, C), call.io)
    y, py = call.output("y", y, x)
    call.run("ttt_step_conv1d", call.dt, B, C, K, int(bool(silu)), px, xs, pw, pb, ps, py, pso)
    return y


def ttt_backward_conv1d(x, weight, bias, d_y, *, silu: bool = False, state=None, lengths=None, d_x=None, d_weight=None,
                        d_bias=None, d_state=None, workspace=None, stream=None):
    """Gradients (d_x, d_weight, d_bias, d_state) of ttt_forward_conv1d given d_y (contiguous [B, N, C]); no
    gradient flows in through state_out. d_state is None without a state, d_bias without a bias."""
    call = _Call("x", x, stream)
    B, N, C, K = _conv_shape(x, weight, 3)
    px, xs = call.rows("x", x, x.shape, C)
    pw, pb = call.need("weight", weight, (C, K)), call.dense("bias", bias, (C,))
    held = (B, K - 1, C)
    ps, pl = call.dense("state", state, held, call.io), call.lengths(lengths, B)
    pdy = call.need("d_y", d_y, x.shape, call.io)
    d_x, pdx = call.output("d_x", d_x, x)
    d_weight, pdw = call.output("d_weight", d_weight, weight)
    pdb = pds = None
    if bias is not None:
        d_bias, pdb = call.output("d_bias", d_bias, bias)
    elif d_bias is not None:
        raise ValueError("d_bias is given without bias")
    if state is not None:
        d_state, pds = call.output("d_state", d_state, state)
    elif d_state is not None:
        raise ValueError("d_state is given without state")
    workspace, pws, nws = call.workspace(workspace, load_library().ttt_backward_conv1d_workspace(call.dt, B, N, C, K))
    call.run("ttt_backward_conv1d", call.dt, B, N, C, K, int(bool(silu)), px, xs, pw, pb, ps, pl, pdy, pdx, pdw, pdb, pds,
             pws, nws)
    return d_x, d_weight, d_bias, d_state


# ---------------------------------------------------------------------- selective state space scan
def _scan_inputs(call, u, delta, A, Bm, Cm, D, delta_bias, z, lead):
    """The C arguments that every direction starts with, and (B, N, C, S, G)."""
    if u.dim() != lead + 1:
        raise ValueError("u must be [B, N, C]" if lead == 2 else "u must be [B, C]")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [C, S]")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != lead + 2:
        raise ValueError("Bm must be [B, N, G, S]" if lead == 2 else "Bm must be [B, G, S]")
    C, S, G = u.shape[-1], A.shape[1], Bm.shape[-2]
    B, N = u.shape[0], u.shape[1] if lead == 2 else 1
    mat = (*u.shape[:-1], G, S)
    args = [*call.rows("u", u, u.shape, C), *call.rows("delta", delta, u.shape, C), call.need("A", A, (C, S)),
            *call.rows("Bm", Bm, mat, G * S), *call.rows("Cm", Cm, mat, G * S), call.dense("D", D, (C,)),
            call.dense("delta_bias", delta_bias, (C,)), *((None, 0) if z is None else call.rows("z", z, u.shape, C))]
    return args, (B, N, C, S, G)


def ttt_forward_selective_scan(u, delta, A, Bm, Cm, D=None, delta_bias=None, z=None, *, softplus: bool = True, h0=None,
                               lengths=None, h_out=None, y=None, workspace=None, stream=None):
    """h = exp(step A) h + step Bm u, y = (Cm . h + D u) * SiLU(z), step = softplus(delta + delta_bias), per channel
    and token. Returns y [B, N, C].

    u, delta, z: [B, N, C] bf16 or fp32; Bm, Cm: [B, N, G, S] (slices of wider rows are read in place); A fp32
    [C, S], S in {8, 16, 32, 64}; D, delta_bias fp32 [C]; h0, h_out: fp32 [B, C, S], the states before the first and
    after the last token; lengths: int32 [B], the tokens of each sequence (y is zero behind them)."""
    call = _Call("u", u, stream)
    args, (B, N, C, S, G) = _scan_inputs(call, u, delta, A, Bm, Cm, D, delta_bias, z, 2)
    ph, pho, pl = call.dense("h0", h0, (B, C, S)), call.dense("h_out", h_out, (B, C, S)), call.lengths(lengths, B)
    y, py = call.output("y", y, u)
    workspace, pws, nws = call.workspace(
        workspace, load_library().ttt_forward_selective_scan_workspace(call.dt, B, N, C, S, G))
    call.run("ttt_forward_selective_scan", call.dt, B, N, C, S, G, int(bool(softplus)), *args, ph, pl, py, pho, pws, nws)
    return y


def ttt_step_selective_scan(u, delta, A, Bm, Cm, D=None, delta_bias=None, z=None, *, h, softplus: bool = True, h_out=None,
                            y=None, stream=None):
    """One token of every sequence: u, delta, z [B, C], Bm, Cm [B, G, S]; h fp32 [B, C, S], updated in place unless
    h_out is given. Returns y [B, C]."""
    call = _Call("u", u, stream)
    args, (B, _, C, S, G) = _scan_inputs(call, u, delta, A, Bm, Cm, D, delta_bias, z, 1)
    ph = call.need("h", h, (B, C, S))
    pho = ph if h_out is None else call.dense("h_out", h_out, (B, C, S))
    y, py = call.output("y", y, u)
    call.run("ttt_step_selective_scan", call.dt, B, C, S, G, int(bool(softplus)), *args, ph, py, pho)
    return y


def ttt_backward_selective_scan(u, delta, A, Bm, Cm, d_y, D=None, delta_bias=None, z=None, *, softplus: bool = True,
                                h0=None, lengths=None, d_u=None, d_delta=None, d_A=None, d_B=None, d_C=None, d_D=None,
                                d_delta_bias=None, d_z=None, d_h0=None, workspace=None, stream=None):
    """Gradients (d_u, d_delta, d_A, d_B, d_C, d_D, d_delta_bias, d_z, d_h0) of ttt_forward_selective_scan given d_y
    (contiguous [B, N, C]); those of inputs that are None are None. No gradient flows in through h_out."""
    call = _Call("u", u, stream)
    args, (B, N, C, S, G) = _scan_inputs(call, u, delta, A, Bm, Cm, D, delta_bias, z, 2)
    ph, pl = call.dense("h0", h0, (B, C, S)), call.lengths(lengths, B)
    pdy = call.need("d_y", d_y, u.shape, call.io)
    outs, ptrs = [], []
    for name, t, of in (("d_u", d_u, u), ("d_delta", d_delta, delta), ("d_A", d_A, A), ("d_B", d_B, Bm), ("d_C", d_C, Cm),
                        ("d_D", d_D, D), ("d_delta_bias", d_delta_bias, delta_bias), ("d_z", d_z, z), ("d_h0", d_h0, h0)):
        if of is None:
            if t is not None:
                raise ValueError(f"{name} is given without its input")
            p = None
        else:
            t, p = call.output(name, t, of)
        outs.append(t)
        ptrs.append(p)
    workspace, pws, nws = call.workspace(
        workspace, load_library().ttt_backward_selective_scan_workspace(call.dt, B, N, C, S, G))
    call.run("ttt_backward_selective_scan", call.dt, B, N, C, S, G, int(bool(softplus)), *args, ph, pl, pdy, *ptrs, pws,
             nws)
    return tuple(outs)
