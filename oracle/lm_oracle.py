"""float64 NumPy oracle of the residual block's operators (include/ttt_lm.h): RMS norm with the residual's addition and an
e4m3 output, dropout, gated linear recurrence, with their gradients. Written out from the definitions, token after token.
TEST INFRASTRUCTURE ONLY.
"""
import numpy as np


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


# ------------------------------------------------------------------------------------ dropout
def philox4x32(counter, key, rounds=10):
    """Four words of a four-word counter under a two-word key, Python integers (Salmon et al., SC'11)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        left, right = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(right >> 32) ^ c[1] ^ k[0], right & 0xFFFFFFFF, (left >> 32) ^ c[3] ^ k[1], left & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def numbers(seed, first, count):
    """The 16-bit numbers of counters first, first + 1, ...: [count, 8]."""
    u = np.uint64
    at = u(first & (2 ** 64 - 1)) + np.arange(count, dtype=u)
    low = u(0xFFFFFFFF)
    c = [at & low, at >> u(32), np.zeros(count, u), np.zeros(count, u)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        left, right = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(right >> u(32)) ^ c[1] ^ u(k[0]), right & low, (left >> u(32)) ^ c[3] ^ u(k[1]), left & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack([(w >> u(s)) & u(0xFFFF) for w in c for s in (0, 16)], -1).astype(np.int64)


def factors(seed, offset, p, M, C):
    """[M, C]: 0 where dropped, otherwise 1 / (1 - p'), p' = T / 65536."""
    T, per = int(np.rint(p * 65536)), -(-C // 8)
    keep = numbers(seed, offset, M * per).reshape(M, per * 8)[:, :C] >= T
    return keep * (65536.0 / (65536 - T))


# ------------------------------------------------------------------------------------ RMS norm
def rmsnorm(s, w, eps):
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w


def rmsnorm_backward(s, w, d_y, eps, d_sum=0.0):
    rstd = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    xhat, g = s * rstd, d_y * w
    d_s = d_sum + rstd * (g - xhat * (g * xhat).mean(-1, keepdims=True))
    return d_s, (d_y * xhat).sum(tuple(range(s.ndim - w.ndim)))


def e4m3(v):
    """The nearest e4m3 number, ties to even: three bits of fraction, in steps of 2^-9 at least, at most 448."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.clip(np.rint(v / step) * step, -448, 448)


# ----------------------------------------------------------------------- gated linear recurrence
def _parts(x, r, i, lam, scale):
    la = -scale * softplus(lam) * sigmoid(r)
    return la, np.exp(la), np.sqrt(-np.expm1(2 * la)), sigmoid(i)


def recurrence(x, r, i, lam, scale=8.0, h0=None, lengths=None):
    """(y, the state after each sequence's last token, the states before each token)."""
    B, N, C = x.shape
    _, a, m, gi = _parts(x, r, i, lam, scale)
    h = np.zeros((B, C)) if h0 is None else h0.copy()
    y, before = np.zeros_like(x), np.zeros_like(x)
    for n in range(N):
        before[:, n] = h
        live = np.ones((B, 1), bool) if lengths is None else (n < np.asarray(lengths))[:, None]
        h = np.where(live, a[:, n] * h + m[:, n] * gi[:, n] * x[:, n], h)
        y[:, n] = np.where(live, h, 0)
    return y, h, before


def recurrence_backward(x, r, i, lam, d_y, scale=8.0, h0=None, lengths=None):
    """{d_x, d_r, d_i, d_lam, d_h0}: the reverse of the forward pass, step for step."""
    B, N, C = x.shape
    la, a, m, gi = _parts(x, r, i, lam, scale)
    _, _, before = recurrence(x, r, i, lam, scale, h0, lengths)
    gr = sigmoid(r)
    z = np.zeros((B, C))
    out = {k: np.zeros_like(x) for k in ("d_x", "d_r", "d_i")}
    d_k = np.zeros(C)
    for n in range(N - 1, -1, -1):
        live = np.ones((B, 1), bool) if lengths is None else (n < np.asarray(lengths))[:, None]
        q = np.where(live, d_y[:, n] + z, 0)
        drive = gi[:, n] * x[:, n]
        d_m, d_a = q * drive, q * before[:, n]
        d_la = d_a * a[:, n] - d_m * a[:, n] ** 2 / m[:, n]
        out["d_x"][:, n] = q * m[:, n] * gi[:, n]
        out["d_i"][:, n] = q * m[:, n] * x[:, n] * gi[:, n] * (1 - gi[:, n])
        out["d_r"][:, n] = d_la * la[:, n] * (1 - gr[:, n])
        d_k += (d_la * -scale * gr[:, n]).sum(0)
        z = np.where(live, a[:, n] * q, z)
    return out | {"d_lam": d_k * sigmoid(lam), "d_h0": z}
