"""The residual block's operators in float64 by torch, on any device, each output with the bound that an fp32 evaluation keeps
to, entry by entry: the first order of what every rounding on the way can do, u = 2^-24 of the value each (an exponential,
a root and a reciprocal by the hardware 2 u). Nothing of the library or of the oracle is used; tests/test_lm_reference.py holds
the values to the oracle. held() of seq_reference.py compares. TEST INFRASTRUCTURE ONLY.
"""
import torch

from seq_reference import U, _d, _live, _sig

ROOT = 2.0 ** -63


# ----------------------------------------------------------------------------------- RMS norm
def _sum(x, residual, factor):
    """s and what it is off by before it is rounded for the output."""
    x = _d(x) if factor is None else torch.where(factor == 0, 0.0, _d(x)) * factor
    off = torch.zeros_like(x) if factor is None else 2 * U * x.abs()  # (the factor's rounding and the product's)
    if residual is None:
        return x, off
    s = x + _d(residual)
    return s, off + U * s.abs()


def _rstd(s, off, eps, depth):
    """1 / sqrt(mean(s^2) + eps) and its relative error: of a square 2 off |s| + u, of sums of `depth` additions, of the
    division by D, of eps's addition, the root and the reciprocal."""
    var = (s * s).mean(-1, keepdim=True)
    off_var = (2 * off * s.abs()).mean(-1, keepdim=True) + (depth + 5) * U * var
    return 1 / torch.sqrt(var + eps), 0.5 * off_var / (var + eps + 1e-300) + 5 * U


def rmsnorm(x, w, eps, depth, residual=None, factor=None):
    """{y, sum: (value, bound)}; x [..., D] with w [D], or [..., H, D] with [H, D]; factor: dropout's."""
    s, off = _sum(x, residual, factor)
    rstd, r = _rstd(s, off, eps, depth)
    y = s * rstd * _d(w)
    return {"y": (y, y.abs() * (r + 3 * U) + off * rstd * _d(w).abs()), "sum": (s, off)}


def rmsnorm_e4m3(x, w, eps, depth, group, residual=None):
    """{scales, deq: (value, bound), sum}: deq is q * scale, within half a step of e4m3 (2^-4 of the value, 2^-10 scales
    below 2^-6 of them) of y."""
    ref = rmsnorm(x, w, eps, depth, residual)
    y, off = (t.unflatten(-1, (-1, group)) for t in ref["y"])
    top, at = y.abs().max(-1)
    off_top = (off + U * y.abs()).amax(-1)
    scale = top.clamp(min=2.0 ** -100) / 448
    step = torch.maximum(y.abs() * 2.0 ** -4, scale[..., None] * 2.0 ** -10)
    deq = y.flatten(-2), (step + (1 + 2.0 ** -4) * (off + 8 * U * y.abs())).flatten(-2) + 2.0 ** -120
    return {"scales": (scale, off_top / 448 + 3 * U * scale), "deq": deq, "sum": ref["sum"]}


def rmsnorm_backward(s, w, d_y, eps, depth, rows_depth, d_sum=None, factor=None):
    """{d_s, d_x, d_weight: (value, bound)}; rows_depth: additions in a parameter's sums."""
    s, w, d_y = _d(s), _d(w), _d(d_y)
    rstd, r = _rstd(s, torch.zeros_like(s), eps, depth)
    xhat = s * rstd
    n = xhat.abs() * (r + U)  # what xhat is off by
    g = d_y * w
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    s2 = mean(g * xhat)
    e2 = mean(g.abs() * n) + (depth + 5) * U * mean((g * xhat).abs())
    inner, size = g - xhat * s2, g.abs() + (xhat * s2).abs()
    d_s, off = rstd * inner, rstd * (inner.abs() * (r + 2 * U) + xhat.abs() * e2 + n * s2.abs() + 4 * U * size)
    if d_sum is not None:
        off = off + U * d_s.abs()
        d_s = d_s + _d(d_sum)
    lead = tuple(range(s.dim() - w.dim()))
    out = {"d_s": (d_s, off + U * d_s.abs()), "d_weight": ((d_y * xhat).sum(lead), (d_y.abs() * n + (rows_depth + 1) * U * (d_y * xhat).abs()).sum(lead))}
    if factor is not None:
        out["d_x"] = d_s * factor, factor * (off + 4 * U * d_s.abs())
    return out


def dropout(x, factor, residual=None):
    return _sum(x, residual, factor)


# ----------------------------------------------------------------------- gated linear recurrence
def recurrence(x, r, i, lam, d_y=None, scale=8.0, h0=None, lengths=None, depth=0):
    """{y, h_out, before} or, given d_y, the gradients: (value, bound). depth: additions in d_lam's sums. before: the states
    before each token.

    Tokens may be taken in runs from zero states, joined by products of decays: a product's rounding is u a token beside
    the decay's own, and each entry goes through four more roundings of its size. The hardware's root takes 1 - a^2 below
    2^-126 as zero: m is off by up to 2^-63 there, and log(a) / m, about -m / 2, by half of that.
    """
    B, N, C = x.shape
    live = _live(lengths, B, N, x.device)[..., None]
    pick = lambda t: None if t is None else torch.where(live, _d(t), 0.0)  # noqa: E731
    x, r, i, d_y, lam = pick(x), pick(r), pick(i), pick(d_y), _d(lam)
    (gr, r_gr), (gi, r_gi) = _sig(r), _sig(i)
    sp = lam.clamp(min=0) + torch.log1p(torch.exp(-lam.abs()))
    la = -scale * sp * gr
    r_la = r_gr + 10 * U                                    # softplus 7 u, two products
    a = torch.exp(la)
    r_a = la.abs() * (r_la + 2 * U) + 3 * U                 # the argument's product and constant, the exponential, its run's product
    w = -torch.expm1(2 * la)
    r_w = torch.where(2 * la > -0.5, r_la + 5 * U, 0.0) + torch.where(2 * la < -0.49, (2 * r_a + U) * a * a / w + U, 0.0)
    m, r_m = torch.sqrt(w), r_w / 2 + 2 * U
    b = torch.where(live, m * gi * x, 0.0)
    flush = torch.where(live, ROOT * gi * x.abs(), 0.0)
    off_b = b.abs() * (r_m + r_gi + 3 * U) + flush
    a, r_a = torch.where(live, a, 1.0), torch.where(live, r_a, 0.0)
    h, H, E = (torch.empty(B, N + 1, C, dtype=torch.float64, device=x.device) for _ in range(3))
    h[:, 0] = 0.0 if h0 is None else _d(h0)
    H[:, 0], E[:, 0] = h[:, 0].abs(), 0.0
    for t in range(N):
        h[:, t + 1] = a[:, t] * h[:, t] + b[:, t]
        H[:, t + 1] = a[:, t] * H[:, t] + b[:, t].abs()
        E[:, t + 1] = a[:, t] * (E[:, t] + r_a[:, t] * H[:, t]) + off_b[:, t] + 2 * U * H[:, t + 1] * live[:, t]
    E = E + 4 * U * H
    if d_y is None:
        y = torch.where(live, h[:, 1:], 0.0), torch.where(live, E[:, 1:], 0.0)
        return {"y": y, "h_out": (h[:, N], E[:, N]), "before": (h[:, :-1], E[:, :-1])}
    q, Q, F = (torch.zeros(B, N, C, dtype=torch.float64, device=x.device) for _ in range(3))
    z, Z, G = (torch.zeros(B, C, dtype=torch.float64, device=x.device) for _ in range(3))
    for t in range(N - 1, -1, -1):
        q[:, t], Q[:, t] = d_y[:, t] + z, d_y[:, t].abs() + Z
        F[:, t] = G + 2 * U * Q[:, t] * live[:, t]
        z, Z = a[:, t] * q[:, t], a[:, t] * Q[:, t]
        G = a[:, t] * F[:, t] + (r_a[:, t] + U) * Z
    F = F + 4 * U * Q
    before, before_size, before_off = h[:, :-1], H[:, :-1], E[:, :-1]
    dx = q * m * gi
    off_dx = F * m * gi + Q * gi * (m * (r_m + r_gi + 2 * U) + ROOT)
    one_gi, off_one_gi = 1 - gi, r_gi * gi + U
    xa = x.abs()
    out = {"d_x": (dx, off_dx), "d_i": (dx * x * one_gi, xa * (off_dx * one_gi + Q * m * gi * (off_one_gi + 2 * U * one_gi)))}
    one, two = a * la * before, a * a * (la / m) * gi * x
    size = a * la.abs() * before_size + two.abs()
    off_in = a * la.abs() * (before_off + before_size * (r_a + r_la + 3 * U)) + two.abs() * (2 * r_a + r_la + r_m + r_gi + 8 * U) + flush
    t_, off_t = q * (one - two), Q * (off_in + 3 * U * size) + F * size
    t_, off_t = torch.where(live, t_, 0.0), torch.where(live, off_t, 0.0)
    size_t = torch.where(live, Q * size, 0.0)
    one_gr, off_one_gr = 1 - gr, r_gr * gr + U
    out["d_r"] = t_ * one_gr, off_t * one_gr + size_t * (off_one_gr + U * one_gr)
    ratio = torch.where(lam < -20, 1.0, torch.sigmoid(lam) / sp)
    out["d_lam"] = t_.sum((0, 1)) * ratio, ratio * (off_t + (depth + 14 + 2 * lam.abs()) * U * size_t).sum((0, 1))
    out["d_h0"] = z, G + 4 * U * Z
    for k in ("d_x", "d_i", "d_r"):
        out[k] = tuple(torch.where(live, v, 0.0) for v in out[k])
    return out
