"""The block operators in float64 by torch, on any device, each output with the bound that an fp32 evaluation keeps to,
entry by entry: the first order of what every rounding on the way can do, u = 2^-24 of the value each (an exponential
and a reciprocal by the hardware 2 u). Nothing of the library or of the oracle is used; tests/test_seq_reference.py
holds the values to the oracle. TEST INFRASTRUCTURE ONLY.

A bound is built from sums of absolute values: what a sum of terms t_i of depth d loses is d u sum |t_i| and what its
terms lose. `depth` arguments are the number of additions that a term can go through.
"""
import torch

U = 2.0 ** -24
TINY = 1e-34  # (exponentials below 2^-126 are zeros)


def _d(t):
    return None if t is None else t.double()


def _live(lengths, B, N, device):
    n = torch.full((B,), N, device=device) if lengths is None else lengths.to(device).long().clamp(0, N)
    return torch.arange(N, device=device)[None, :] < n[:, None]


def _sig(x):
    """sigmoid, and its relative error: of exp(-x) (2 |x| + 2) u times its share of the sum, then a sum and a reciprocal."""
    s = torch.sigmoid(x)
    return s, ((2 * x.abs() + 2) * (1 - s) + 3) * U


def _silu(x):
    """x sigmoid(x) and its relative error; its derivative and its absolute error."""
    s, r = _sig(x)
    one = 1 + x.abs() * (1 - s)
    return x * s, r + U, s * (1 + x * (1 - s)), s * (r * (1 + x.abs()) + 4 * U * one)


# ---------------------------------------------------------------------------------- layer norm
def layernorm(x, w, b, d_y, eps, depth, rows_depth):
    """{y, d_x, d_weight, d_bias: (value, bound)}; x [..., D] with w [D], or [..., H, D] with [H, D]. The
    mean of an fp32 row is its first element and the mean of what the others differ from it, kept as two numbers. depth: additions in a row's sums; rows_depth: in a parameter's."""
    fp32 = x.dtype == torch.float32
    x, w, b, d_y = _d(x), _d(w), _d(b), _d(d_y)
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    e = (x - x[..., :1]) if fp32 else x
    c = x - mean(x)
    off = (1 + fp32) * U * c.abs() + (depth + 3) * U * mean(e.abs())
    var = mean(c * c)
    off_var = 2 * mean(c.abs() * off) + (depth + 4) * U * var
    rstd = 1 / torch.sqrt(var + eps)
    r = 0.5 * off_var / (var + eps) + 4 * U
    xhat = c * rstd
    n = rstd * off + xhat.abs() * (r + U)
    y = xhat * w + (0 if b is None else b)
    out = {"y": (y, w.abs() * n + 2 * U * ((xhat * w).abs() + (0 if b is None else b.abs())))}
    if d_y is None:
        return out
    g = d_y * w
    s1, s2 = mean(g), mean(g * xhat)
    e1 = (depth + 4) * U * mean(g.abs())
    e2 = mean(g.abs() * n) + (depth + 4) * U * mean((g * xhat).abs())
    inner = g - s1 - xhat * s2
    size = g.abs() + s1.abs() + (xhat * s2).abs()
    out["d_x"] = rstd * inner, rstd * (inner.abs() * (r + 2 * U) + e1 + xhat.abs() * e2 + n * s2.abs() + 4 * U * size)
    lead = tuple(range(x.dim() - w.dim()))
    out["d_weight"] = (d_y * xhat).sum(lead), (d_y.abs() * n + (rows_depth + 1) * U * (d_y * xhat).abs()).sum(lead)
    out["d_bias"] = d_y.sum(lead), rows_depth * U * d_y.abs().sum(lead)
    return out


# ------------------------------------------------------------------- short causal convolution
def conv1d(x, w, b, d_y=None, silu=False, state=None, lengths=None, rows_depth=0):
    """{y, d_x, d_weight, d_bias, d_state: (value, bound)}."""
    B, N, C = x.shape
    K = w.shape[1]
    live = _live(lengths, B, N, x.device)[..., None]
    x, w, b = torch.where(live, _d(x), 0.0), _d(w), _d(b)
    before = torch.zeros(B, K - 1, C, dtype=torch.float64, device=x.device) if state is None else _d(state)
    line = torch.cat([before, x], 1)
    pre = torch.zeros_like(x) if b is None else b.expand_as(x).clone()
    size = pre.abs()
    for k in range(K):
        pre, size = pre + w[:, k] * line[:, k:k + N], size + (w[:, k] * line[:, k:k + N]).abs()
    off = (K + 1) * U * size
    if silu:
        y, r, slope, off_slope = _silu(pre)
        out = {"y": (torch.where(live, y, 0.0), torch.where(live, 1.1 * off + y.abs() * r, 0.0))}
    else:
        slope, off_slope = torch.ones_like(pre), torch.zeros_like(pre)
        out = {"y": (torch.where(live, pre, 0.0), torch.where(live, off, 0.0))}
    if d_y is None:
        return out
    g = torch.where(live, _d(d_y), 0.0)
    d, off_d = g * slope, g.abs() * (off_slope + (0.5 * off if silu else 0.0)) + U * (g * slope).abs()
    d_line, off_line = torch.zeros_like(line), torch.zeros_like(line)
    dw, off_w = torch.zeros_like(w), torch.zeros_like(w)
    for k in range(K):
        d_line[:, k:k + N] += w[:, k] * d
        off_line[:, k:k + N] += w[:, k].abs() * (off_d + (K + 1) * U * d.abs())
        part = line[:, k:k + N]
        dw[:, k] = (d * part).sum((0, 1))
        off_w[:, k] = (off_d * part.abs() + (rows_depth + 1) * U * (d * part).abs()).sum((0, 1))
    out["d_x"] = d_line[:, K - 1:], off_line[:, K - 1:]
    out["d_state"] = d_line[:, :K - 1], off_line[:, :K - 1]
    out["d_weight"] = dw, off_w
    out["d_bias"] = d.sum((0, 1)), (off_d + rows_depth * U * d.abs()).sum((0, 1))
    return out


# ---------------------------------------------------------------------- selective state space scan
def scan(u, delta, A, Bm, Cm, D=None, delta_bias=None, z=None, d_y=None, softplus=True, h0=None, lengths=None, tokens=1, depth=0):
    """{y, h_out, or the gradients: (value, bound)}. tokens: of a segment (a sum of as many steps gives its decay);
    depth: additions in a parameter's sums."""
    B, N, C = u.shape
    S, G, dev = A.shape[1], Bm.shape[2], u.device
    blocks = (C // G + 63) // 64
    live = _live(lengths, B, N, dev)
    pick = lambda t: None if t is None else torch.where(live.view(B, N, *[1] * (t.dim() - 2)), _d(t), 0.0)  # noqa: E731
    u, z, d_y, A, D = pick(u), pick(z), pick(d_y), _d(A), (torch.zeros(C, dtype=torch.float64, device=dev) if D is None else _d(D))
    raw = pick(delta) + (0 if delta_bias is None else _d(delta_bias))
    off_raw = U * raw.abs()
    if softplus:
        log1p = torch.log1p(torch.exp(-raw.abs()))
        dt, s = raw.clamp(min=0) + log1p, torch.sigmoid(raw)
        off_dt = s * off_raw + log1p * (2 * raw.abs() + 8) * U + 2 * U * dt
        slope, off_slope = s, s * ((2 * raw.abs() + 6) * U + (1 - s) * off_raw)
    else:
        dt, off_dt, slope, off_slope = raw, off_raw, torch.ones_like(raw), torch.zeros_like(raw)
    dt, off_dt = (torch.where(live[..., None], t, 0.0)[..., None] for t in (dt, off_dt))  # [B, N, C, 1]
    wide = lambda m: pick(m).repeat_interleave(C // G, 2)  # noqa: E731
    Bc, Cc = wide(Bm), wide(Cm)                            # [B, N, C, S]
    a = torch.exp(dt * A)
    off_a = (A.abs() * (off_dt + (3 + tokens) * U * dt.abs()) + 3 * U) * live[..., None, None]  # relative
    b = dt * u[..., None] * Bc
    off_b = (u[..., None] * Bc).abs() * (off_dt + 2 * U * dt.abs())
    # States h, of absolute values H, and what they are off by, E: before the first token and after each.
    h, H, E = (torch.empty(B, N + 1, C, S, dtype=torch.float64, device=dev) for _ in range(3))
    h[:, 0] = 0.0 if h0 is None else _d(h0)
    H[:, 0], E[:, 0] = h[:, 0].abs(), 0.0
    size_b = b.abs()
    for t in range(N):
        torch.addcmul(b[:, t], a[:, t], h[:, t], out=h[:, t + 1])
        torch.addcmul(size_b[:, t], a[:, t], H[:, t], out=H[:, t + 1])
        torch.addcmul(off_b[:, t], a[:, t], torch.addcmul(E[:, t], off_a[:, t], H[:, t]), out=E[:, t + 1])
        E[:, t + 1].add_(H[:, t + 1], alpha=2 * U)
    Ca = Cc.abs()
    o = (Cc * h[:, 1:]).sum(-1) + D * u
    size_o = (Ca * H[:, 1:]).sum(-1) + (D * u).abs()
    off_o = (Ca * E[:, 1:]).sum(-1) + (S / 2 + 3) * U * size_o
    if z is None:
        gate, r_gate = torch.ones_like(o), torch.zeros_like(o)
    else:
        gate, r_gate, gate_slope, off_gate_slope = _silu(z)
    if d_y is None:
        y = o * gate * live[..., None]
        off = (gate.abs() * off_o + size_o * gate.abs() * (r_gate + 2 * U)) * live[..., None]
        return {"y": (y, off), "h_out": (h[:, N].clone(), E[:, N].clone())}
    v, r_v = d_y * gate, r_gate + 2 * U                  # [B, N, C]; relative
    # q_n = v C + a_{n+1} q_{n+1}, of absolute values Q, and what it is off by, F; and what a_n of it is.
    vC, size_vC = v[..., None] * Cc, v.abs()[..., None] * Ca
    q, Q, F = (torch.zeros(B, N + 1, C, S, dtype=torch.float64, device=dev) for _ in range(3))  # q[:, n]: after token n - 1
    qa, Qa, Fa = (torch.zeros(B, C, S, dtype=torch.float64, device=dev) for _ in range(3))
    off_vC = size_vC * (r_v + U)[..., None]
    for t in range(N - 1, -1, -1):
        torch.add(vC[:, t], qa, out=q[:, t + 1])
        torch.add(size_vC[:, t], Qa, out=Q[:, t + 1])
        torch.add(off_vC[:, t], Fa, out=F[:, t + 1])
        F[:, t + 1].add_(Q[:, t + 1], alpha=2 * U)
        qa, Qa = a[:, t] * q[:, t + 1], a[:, t] * Q[:, t + 1]
        Fa = a[:, t] * F[:, t + 1] + (off_a[:, t] + U) * Qa
    out = {"d_h0": (qa, Fa)}
    q, Q, F = q[:, 1:], Q[:, 1:], F[:, 1:]
    before, before_size, before_off = h[:, :-1], H[:, :-1], E[:, :-1]
    Ba = Bc.abs()
    qB, size_qB = (q * Bc).sum(-1), (Q * Ba).sum(-1)
    off_qB = (F * Ba).sum(-1) + (S + 4) * U * size_qB
    dt3, off3 = dt[..., 0], off_dt[..., 0]
    Dv = (D * v).abs()
    out["d_u"] = (dt3 * qB + D * v, dt3.abs() * off_qB + off3 * size_qB + Dv * (r_v + 2 * U) + 2 * U * (dt3.abs() * size_qB + Dv))
    g, size_g = q * a * before, Q * a * before_size
    off_g = a * (F * before_size + Q * before_off) + (off_a + 3 * U) * size_g
    step = (g * A).sum(-1) + u * qB
    size_step = (size_g * A.abs()).sum(-1) + u.abs() * size_qB
    off_step = (off_g * A.abs()).sum(-1) + u.abs() * off_qB + (S + 6) * U * size_step
    dd, off_dd = step * slope, off_step * slope.abs() + size_step * off_slope + 2 * U * size_step * slope.abs()
    out["d_delta"] = dd, off_dd
    out["d_delta_bias"] = dd.sum((0, 1)), (off_dd + depth * U * dd.abs()).sum((0, 1))
    out["d_A"] = (g * dt).sum((0, 1)), (off_g * dt.abs() + size_g * (off_dt + (depth + 1) * U * dt.abs())).sum((0, 1))
    out["d_D"] = (v * u).sum((0, 1)), (v * u).abs().mul(r_v + (depth + 1) * U).sum((0, 1))
    per_group = lambda t: t.view(B, N, G, C // G, S).sum(3)  # noqa: E731
    ua = u.abs()[..., None]
    out["d_B"] = (per_group(q * dt * u[..., None]),
                  per_group(ua * (F * dt.abs() + Q * off_dt + (blocks + 10) * U * Q * dt.abs())))
    va = v.abs()[..., None]
    out["d_C"] = (per_group(v[..., None] * h[:, 1:]),
                  per_group(va * E[:, 1:] + va * H[:, 1:] * (r_v + (blocks + 9) * U)[..., None]))
    if z is not None:
        out["d_z"] = (d_y * o * gate_slope, d_y.abs() * (off_o * gate_slope.abs() + size_o * (off_gate_slope + 3 * U * gate_slope.abs())))
    return out


def held(name, got, ref):
    """got (the library's tensor) to ref = (value, bound) and its type's own rounding, half a step; returns the worst
    share of the bound. Every entry has to be finite."""
    value, bound = ref
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    bound = bound + (torch.finfo(got.dtype).eps / 2) * (value.abs() + bound) + TINY
    share = (got.double() - value).abs() / bound
    worst = float(share.max()) if share.numel() else 0.0
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound at {int(share.argmax())} of {tuple(got.shape)}"
    return worst
