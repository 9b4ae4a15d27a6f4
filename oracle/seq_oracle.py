"""fp64 CPU oracle of the block operators: layer norm, the short causal convolution and the selective
state space scan, each with its gradients.

TEST INFRASTRUCTURE ONLY: only tests/ may use it. It shares no code with the HIP library and does not
import the package.

What it computes, for arrays [B, N, C] of tokens and channels (layer norm: the last axis):
  layer norm   y = (x - mean) / sqrt(var + eps) w + b, var the population variance;
  convolution  pre[n] = b + sum_k w[:, k] x[n - (K - 1) + k], x before token 0 from the state or zero,
               y = pre or pre sigmoid(pre);
  scan         step = softplus(delta + bias), h = exp(step A) h + step B u, y = (C . h + D u) z sigmoid(z).
Sequences end at their length: the tokens behind it have y = 0 and take no part in anything.

Parity status: pinned by tests/test_oracle_pins_seq.py (closed forms, torch's layer norm and
convolution, brute force on tiny inputs, every gradient against central differences).
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def _dsilu(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


def _lengths(lengths, B, N):
    return [N] * B if lengths is None else [int(min(max(n, 0), N)) for n in lengths]


# ---------------------------------------------------------------------------------- layer norm
def layernorm(x, w, b, eps):
    """x [..., D] with w, b [D], or [..., H, D] with [H, D]."""
    x, w, b = _f64(x), _f64(w), _f64(b)
    mean = x.mean(-1, keepdims=True)
    var = ((x - mean) ** 2).mean(-1, keepdims=True)
    y = (x - mean) / np.sqrt(var + eps) * w
    return y if b is None else y + b


def layernorm_backward(x, w, dy, eps):
    x, w, dy = _f64(x), _f64(w), _f64(dy)
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    xhat = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdims=True) - xhat * (g * xhat).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - w.ndim))
    return dx, (dy * xhat).sum(lead), dy.sum(lead)


# ------------------------------------------------------------------- short causal convolution
def conv1d(x, w, b, silu, state=None, lengths=None):
    """Returns y [B, N, C] and the state after each sequence's last token [B, K - 1, C]."""
    x, w, b, state = _f64(x), _f64(w), _f64(b), _f64(state)
    B, N, C = x.shape
    K = w.shape[1]
    y, out = np.zeros((B, N, C)), np.zeros((B, K - 1, C))
    for i, n in enumerate(_lengths(lengths, B, N)):
        line = np.concatenate([np.zeros((K - 1, C)) if state is None else state[i], x[i, :n]])
        pre = np.zeros((n, C)) if b is None else np.broadcast_to(b, (n, C)).copy()
        for k in range(K):
            pre += w[:, k] * line[k:k + n]
        y[i, :n] = pre * sigmoid(pre) if silu else pre
        out[i] = line[n:]
    return y, out


def conv1d_backward(x, w, b, silu, dy, state=None, lengths=None):
    """Returns dx, dw, db, dstate."""
    x, w, b, state, dy = _f64(x), _f64(w), _f64(b), _f64(state), _f64(dy)
    B, N, C = x.shape
    K = w.shape[1]
    dx, dw, db, ds = np.zeros((B, N, C)), np.zeros((C, K)), np.zeros(C), np.zeros((B, K - 1, C))
    for i, n in enumerate(_lengths(lengths, B, N)):
        line = np.concatenate([np.zeros((K - 1, C)) if state is None else state[i], x[i, :n]])
        dpre = dy[i, :n]
        if silu:
            pre = np.zeros((n, C)) if b is None else np.broadcast_to(b, (n, C)).copy()
            for k in range(K):
                pre += w[:, k] * line[k:k + n]
            dpre = dpre * _dsilu(pre)
        dline = np.zeros_like(line)
        for k in range(K):
            dline[k:k + n] += w[:, k] * dpre
            dw[:, k] += (dpre * line[k:k + n]).sum(0)
        db += dpre.sum(0)
        ds[i], dx[i, :n] = dline[:K - 1], dline[K - 1:]
    return dx, dw, db, ds


# ---------------------------------------------------------------------- selective state space scan
def _scan_inputs(u, delta, A, Bm, Cm, D, dbias, z, sp):
    u, delta, A, Bm, Cm, D, dbias, z = map(_f64, (u, delta, A, Bm, Cm, D, dbias, z))
    C, G = u.shape[2], Bm.shape[2]
    raw = delta if dbias is None else delta + dbias
    dt = softplus(raw) if sp else raw
    rep = lambda m: np.repeat(m, C // G, axis=2)  # noqa: E731
    return u, raw, dt, A, rep(Bm), rep(Cm), np.zeros(C) if D is None else D, z


def scan(u, delta, A, Bm, Cm, D=None, dbias=None, z=None, sp=True, h0=None, lengths=None):
    """Returns y [B, N, C] and the end states [B, C, S]."""
    u, _, dt, A, Bc, Cc, D, z = _scan_inputs(u, delta, A, Bm, Cm, D, dbias, z, sp)
    B, N, C = u.shape
    h = np.zeros((B, C, A.shape[1])) if h0 is None else _f64(h0).copy()
    y = np.zeros((B, N, C))
    for i, n in enumerate(_lengths(lengths, B, N)):
        for t in range(n):
            h[i] = np.exp(dt[i, t][:, None] * A) * h[i] + (dt[i, t] * u[i, t])[:, None] * Bc[i, t]
            y[i, t] = (Cc[i, t] * h[i]).sum(-1) + D * u[i, t]
            if z is not None:
                y[i, t] *= z[i, t] * sigmoid(z[i, t])
    return y, h


def scan_backward(u, delta, A, Bm, Cm, dy, D=None, dbias=None, z=None, sp=True, h0=None, lengths=None):
    """Returns a dict of the gradients d_u, d_delta, d_A, d_B, d_C, d_D, d_delta_bias, d_z, d_h0."""
    G, dy = np.shape(Bm)[2], _f64(dy)
    u, raw, dt, A, Bc, Cc, D, z = _scan_inputs(u, delta, A, Bm, Cm, D, dbias, z, sp)
    B, N, C = u.shape
    S = A.shape[1]
    start = np.zeros((B, C, S)) if h0 is None else _f64(h0)
    g = {k: np.zeros((B, N, C)) for k in ("d_u", "d_delta", "d_z")}
    dB, dC = np.zeros((B, N, C, S)), np.zeros((B, N, C, S))
    g |= {"d_A": np.zeros((C, S)), "d_D": np.zeros(C), "d_delta_bias": np.zeros(C), "d_h0": np.zeros((B, C, S))}
    for i, n in enumerate(_lengths(lengths, B, N)):
        hs = [start[i]]
        for t in range(n):
            hs.append(np.exp(dt[i, t][:, None] * A) * hs[-1] + (dt[i, t] * u[i, t])[:, None] * Bc[i, t])
        q = np.zeros((C, S))  # gradient of the state after token t, from the tokens behind it
        for t in range(n - 1, -1, -1):
            v, out = dy[i, t], (Cc[i, t] * hs[t + 1]).sum(-1) + D * u[i, t]
            if z is not None:
                g["d_z"][i, t] = v * out * _dsilu(z[i, t])
                v = v * z[i, t] * sigmoid(z[i, t])
            q = q + v[:, None] * Cc[i, t]
            a = np.exp(dt[i, t][:, None] * A)
            dB[i, t], dC[i, t] = q * (dt[i, t] * u[i, t])[:, None], v[:, None] * hs[t + 1]
            qb = (q * Bc[i, t]).sum(-1)
            g["d_u"][i, t] = dt[i, t] * qb + D * v
            g["d_D"] += v * u[i, t]
            d_dt = u[i, t] * qb + (q * a * hs[t] * A).sum(-1)
            g["d_A"] += q * a * hs[t] * dt[i, t][:, None]
            g["d_delta"][i, t] = d_dt * sigmoid(raw[i, t]) if sp else d_dt
            q = q * a
        g["d_h0"][i] = q
    g["d_delta_bias"] = g["d_delta"].sum((0, 1))
    g["d_B"] = dB.reshape(B, N, G, C // G, S).sum(3)
    g["d_C"] = dC.reshape(B, N, G, C // G, S).sum(3)
    return g
