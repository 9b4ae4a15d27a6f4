"""What is measured of the operators of a recurrent language block: the RMS norm with the residual's addition
(with dropout on the branch, or an output in 8 bits), dropout, and the gated linear recurrence, each in its directions.

`own` chooses between the operators' plain forms (elementary torch operations in 32 bits, rounded once at
the end) and the library's entry points; both take what `prepare` gives. `exact` computes the same outputs
in 64 bits from the operators' definitions, the gradients by differentiation.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DECAY = 8.0  # the recurrence's scale of its decay's exponent
KEPT = 64    # tokens between the states that a recurrence's forward pass keeps for the backward pass
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ the cases
def _norm(name, direction, M, H, D, dtype, residual=True, p=0.0, group=0, sliced=False):
    return {"name": name, "op": "rmsnorm", "direction": direction, "M": M, "H": H, "D": D, "dtype": dtype,
            "residual": residual, "p": p, "group": group, "sliced": sliced}


def _drop(name, direction, M, C, dtype, p, residual=False):
    return {"name": name, "op": "dropout", "direction": direction, "M": M, "C": C, "dtype": dtype, "p": p,
            "residual": residual}


def _rec(name, direction, B, N, C, dtype, state=False, ragged=False, kept=False):
    return {"name": name, "op": "recurrence", "direction": direction, "B": B, "N": N, "C": C, "dtype": dtype,
            "state": state, "ragged": ragged, "kept": kept}


def listed():
    return [
        # one new token of each of 16 sequences at the language layers' width (12 heads x 64), normed into 8 bits for
        # a projection in 8 bits, one scale a token: latency
        _norm("rmsnorm_e4m3_tokens", "e4m3", 16, 1, 768, "bf16"),
        # a prompt of 16384 tokens at twice that width, a scale for every 128 channels
        _norm("rmsnorm_e4m3_prompt", "e4m3", 16384, 1, 1536, "bf16", group=128),
        # a training step at 4 x 8192 tokens: the branch's dropout, the residual's addition and the norm at once
        _norm("rmsnorm_fwd_train", "forward", 4 * 8192, 1, 768, "bf16", p=0.1),
        # and back, the residual stream's own gradient joined in
        _norm("rmsnorm_bwd_train", "backward", 4 * 8192, 1, 768, "bf16", p=0.1),
        # fp32 training at an odd width and token count: no vector access fits its rows
        _norm("rmsnorm_bwd_odd", "backward", 1537, 1, 1001, "fp32"),
        # the branch of 64 images of 14 x 14 tokens, width 6 x 64, dropped and added to the residual stream
        _drop("dropout_fwd_images", "forward", 64 * 196, 384, "bf16", 0.1, residual=True),
        # the gradient of an odd width in fp32
        _drop("dropout_bwd_odd", "backward", 1537, 1001, "fp32", 0.25),
        # the recurrence over prompts of the language layer's shape, its end state kept
        _rec("recurrence_fwd_prompt", "forward", 4, 8192, 768, "bf16"),
        # a padded fp32 batch of unequal prompts that continue earlier ones
        _rec("recurrence_fwd_ragged", "forward", 3, 1999, 1000, "fp32", state=True, ragged=True),
        # a training step's way back, the states that the way forward kept at hand
        _rec("recurrence_bwd_train", "backward", 4, 8192, 768, "bf16", kept=True),
        # a small fp32 training step at odd sizes that keeps nothing
        _rec("recurrence_bwd_odd", "backward", 2, 333, 193, "fp32", state=True),
        # one new token for each of 64 sequences
        _rec("recurrence_step", "step", 64, 1, 1536, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["rmsnorm", "rmsnorm", "dropout", "recurrence", "recurrence"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        p = rng.choice([0.0, 0.1, 0.25, round(rng.uniform(0.01, 0.9), 3)])
        if op == "rmsnorm":
            direction = rng.choice(["forward", "e4m3", "backward"])
            H = rng.choice([1, 1, 1, 6, 12])
            group = rng.choice([0, 32, 64, 128]) if direction == "e4m3" else 0
            D = _log_int(rng, 33, 4096) if H == 1 else rng.choice([16, 32, 64, 128])
            D = D if H > 1 else (D + group - 1) // group * group if group else D if rng.random() < 0.4 else (D + 15) // 16 * 16
            group = group if group and D % group == 0 else 0
            residual = H == 1 and rng.random() < 0.7
            c = _norm("", direction, _log_int(rng, 1, 40000), H, D, dtype, residual,
                      p if residual and direction != "e4m3" else 0.0, group, rng.random() < 0.3)
        elif op == "dropout":
            C = _log_int(rng, 17, 4096)
            c = _drop("", rng.choice(["forward", "backward"]), _log_int(rng, 1, 40000), C if rng.random() < 0.4 else (C + 15) // 16 * 16,
                      dtype, max(p, 0.05), rng.random() < 0.5)
        else:
            direction = rng.choice(["forward", "backward", "step"])
            step = direction == "step"
            C = _log_int(rng, 17, 2560)
            C = C if rng.random() < 0.4 else (C + 15) // 16 * 16
            c = _rec("", direction, _log_int(rng, 1, 256 if step else 8), 1 if step else _log_int(rng, 1, 16384), C, dtype,
                     rng.random() < 0.5, not step and rng.random() < 0.4, direction == "backward" and rng.random() < 0.5)
        del c["name"]
        if work(c)["bytes"] <= most:
            return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rmsnorm":
        M, width, add, drop = case["M"], case["H"] * case["D"], int(case["residual"]), int(case["p"] > 0)
        n = M * width
        if case["direction"] == "backward":
            return {"bytes": (3 + add + drop) * n * e + 8 * width, "flops": (12 + 15 * drop) * n}
        if case["direction"] == "e4m3":
            scales = 4 * n // (case["group"] or case["D"])
            return {"bytes": (1 + 2 * add) * n * e + n + scales + 4 * width, "flops": 10 * n}
        return {"bytes": (2 + 2 * add) * n * e + 4 * width, "flops": (6 + 15 * drop) * n}
    if case["op"] == "dropout":
        n = case["M"] * case["C"]
        return {"bytes": (2 + int(case["residual"] and case["direction"] == "forward")) * n * e + 16, "flops": 15 * n}
    B, N, C = case["B"], case["N"], case["C"]
    state = 4 * B * C
    if case["direction"] == "step":
        return {"bytes": 4 * B * C * e + 2 * state + 4 * C, "flops": 25 * B * C}
    if case["direction"] == "backward":
        kept = 4 * B * C * ((N + KEPT - 1) // KEPT) if case["kept"] else 0
        return {"bytes": 7 * B * N * C * e + (2 * state if case["state"] else 0) + kept + 8 * C, "flops": 55 * B * N * C}
    return {"bytes": 4 * B * N * C * e + (2 if case["state"] else 1) * state + 4 * C, "flops": 25 * B * N * C}


# ---------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale + mean).to(dtype)

    s = {"case": dict(case)}
    if case["op"] != "recurrence" and case["p"] > 0:
        s["rng"] = torch.randint(0, 1 << 40, (2,), device="cuda", generator=gen)  # the seed, and how far it has been used
    if case["op"] == "dropout":
        M, C = case["M"], case["C"]
        if case["direction"] == "backward":
            s["d_y"] = normal(M, C, dtype=dt)
            return s
        s["x"] = normal(M, C, scale=0.5, dtype=dt)
        if case["residual"]:
            s["residual"] = normal(M, C, scale=2.0, dtype=dt)
        return s
    if case["op"] == "rmsnorm":
        M, H, D = case["M"], case["H"], case["D"]
        shape = (M, H, D) if H > 1 else (M, D)
        # activations of a residual stream: channels of unequal size
        size = torch.exp(normal(H * D, scale=0.5))
        x = (normal(M, H * D) * size).to(dt)
        if case["sliced"]:
            rows = torch.zeros(M, 3 * H * D, device="cuda", dtype=dt)
            rows[:, :H * D] = x
            x = rows[:, :H * D]
        s["x"] = x.view(shape)
        s["weight"] = normal(*shape[1:], scale=0.2, mean=1.0)
        if case["direction"] == "backward":
            s["d_y"] = normal(*shape, dtype=dt)
            if case["residual"]:
                s["d_sum"] = normal(*shape, dtype=dt)
        elif case["residual"]:
            s["residual"] = normal(*shape, scale=2.0, dtype=dt)
        return s
    B, N, C, step = case["B"], case["N"], case["C"], case["direction"] == "step"
    lead = (B,) if step else (B, N)
    if case["ragged"]:
        lengths = torch.randint(0, N + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
        lengths[0] = N  # a batch is padded to its longest sequence
        s["lengths"] = lengths
    gates = normal(*lead, 2 * C, dtype=dt)  # both gates' projection
    s["x"], s["r"], s["i"] = normal(*lead, C, dtype=dt), gates[..., :C], gates[..., C:]
    # decays of 0.9 to 0.999 a token where the gate is wide open
    decay = torch.rand(C, device="cuda", generator=gen) * 0.099 + 0.9
    s["lam"] = torch.log(torch.expm1(-torch.log(decay) / DECAY))
    if case["state"] or step:
        s["h"] = normal(B, C, scale=0.5)
    if case["direction"] == "backward":
        s["d_y"] = normal(B, N, C, dtype=dt)
        if case["kept"]:  # the states before tokens 0, KEPT, 2 KEPT, ..., as the way forward left them
            h = _rec_parts(s)[-1]
            h0 = s["h"][:, None] if "h" in s else torch.zeros(B, 1, C, device="cuda")
            s["states"] = torch.cat([h0, h[:, KEPT - 1:N - 1:KEPT]], 1).contiguous()
    else:
        s["h_out"] = torch.empty(B, C, device="cuda")
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    return _PLAIN[case["op"], case["direction"]](state)


# -------------------------------------------------------------------------- the library's calls
def _own(s):
    import test_sequence_layers_amd as T

    case = s["case"]
    op, direction, p = case["op"], case["direction"], case.get("p", 0.0)
    if op == "dropout":
        if direction == "forward":
            return {"y": T.ttt_forward_dropout(s["x"], p, s["rng"], residual=s.get("residual"))}
        return {"d_x": T.ttt_backward_dropout(s["d_y"], p, s["rng"])}
    if op == "rmsnorm":
        if direction == "backward":
            got = T.ttt_backward_rmsnorm(s["x"], s["weight"], s["d_y"], EPS, d_sum=s.get("d_sum"), p=p, rng=s.get("rng"))
            return {k: v for k, v in zip(("d_s", "d_x", "d_weight"), got) if v is not None}
        if direction == "e4m3":
            got = T.ttt_forward_rmsnorm_e4m3(s["x"], s["weight"], EPS, residual=s.get("residual"), group=case["group"])
            return dict(zip(("y", "scales", "sum"), got))
        got = T.ttt_forward_rmsnorm(s["x"], s["weight"], EPS, residual=s.get("residual"), p=p, rng=s.get("rng"))
        return dict(zip(("y", "sum"), got)) if case["residual"] else {"y": got}
    mats = (s["x"], s["r"], s["i"], s["lam"])
    if direction == "step":
        y = T.ttt_step_gated_recurrence(*mats, scale=DECAY, h=s["h"], h_out=s["h_out"])
        return {"y": y, "h_out": s["h_out"]}
    more = {"scale": DECAY, "h0": s.get("h"), "lengths": s.get("lengths")}
    if direction == "forward":
        y = T.ttt_forward_gated_recurrence(*mats, h_out=s["h_out"], **more)
        return {"y": y, "h_out": s["h_out"]}
    got = T.ttt_backward_gated_recurrence(*mats, s["d_y"], states=s.get("states"), **more)
    return {k: v for k, v in zip(("d_x", "d_r", "d_i", "d_lam", "d_h0"), got) if v is not None}


# ------------------------------------------------------------------------------- the plain forms
_M0, _M1, _W0, _W1, _LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _keep(rng, p, M, C):
    """[M, C] of ones and zeros: Philox 4x32 in 10 rounds, keyed by the seed, at counter offset + m ceil(C / 8) + c / 8;
    its four words are eight 16-bit numbers, the lower halves first, and channel c is kept where number c % 8 is not below
    65536 p. (64-bit products wrap; their upper halves are masked out.)"""
    per = (C + 7) // 8
    at = rng[1] + torch.arange(M * per, device="cuda")
    c0, c1 = at & _LOW, (at >> 32) & _LOW
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = rng[0] & _LOW, (rng[0] >> 32) & _LOW
    for _ in range(10):
        p0, p1 = c0 * _M0, c2 * _M1
        c0, c1, c2, c3 = ((p1 >> 32) & _LOW) ^ c1 ^ k0, p1 & _LOW, ((p0 >> 32) & _LOW) ^ c3 ^ k1, p0 & _LOW
        k0, k1 = (k0 + _W0) & _LOW, (k1 + _W1) & _LOW
    words = torch.stack([c0, c1, c2, c3], -1)
    u16 = torch.stack([words & 0xFFFF, words >> 16], -1).view(M, per * 8)[:, :C]
    return (u16 >= round(p * 65536)).float()


def _dropped(s, x):
    """x in 32 bits, dropped and scaled where the case drops."""
    case, x = s["case"], x.float()
    if case["p"] == 0:
        return x
    return x * _keep(s["rng"], case["p"], case["M"], x.shape[-1]) * (65536 / (65536 - round(case["p"] * 65536)))


def _plain_dropout(s):
    y = _dropped(s, s["x"])
    return {"y": (y + s["residual"].float() if "residual" in s else y).to(s["x"].dtype)}


def _plain_dropout_backward(s):
    return {"d_x": _dropped(s, s["d_y"]).to(s["d_y"].dtype)}


def _plain_normed(s):
    total = s["residual"].float() + _dropped(s, s["x"]) if "residual" in s else s["x"].float()
    rstd = torch.rsqrt((total * total).mean(-1, keepdim=True) + EPS)
    return total * rstd * s["weight"], total


def _with_sum(s, out, total):
    if "residual" in s:
        out["sum"] = total.to(s["x"].dtype)
    return out


def _plain_rmsnorm(s):
    y, total = _plain_normed(s)
    return _with_sum(s, {"y": y.to(s["x"].dtype)}, total)


def _plain_rmsnorm_e4m3(s):
    y, total = _plain_normed(s)
    groups = y.unflatten(-1, (-1, s["case"]["group"] or s["case"]["D"]))
    scales = groups.abs().amax(-1).clamp(min=2.0 ** -100) / 448
    q = (groups / scales[..., None]).flatten(-2).to(torch.float8_e4m3fn)
    return _with_sum(s, {"y": q, "scales": scales}, total)


def _plain_rmsnorm_backward(s):
    x, dy = s["x"].float(), s["d_y"].float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat, g = x * rstd, dy * s["weight"]
    ds = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if "d_sum" in s:
        ds = ds + s["d_sum"].float()
    out = {"d_s": ds.to(s["x"].dtype), "d_weight": (dy * xhat).sum(0)}
    if s["case"]["p"] > 0:
        out["d_x"] = _dropped(s, ds).to(s["x"].dtype)
    return out


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _recurrence(a, b):
    """h[t] = a[t] h[t - 1] + b[t] along dim 1 for all t at once: pairs of steps are joined, then pairs of pairs."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _rec_parts(s):
    """x and the gates in 32 bits, the decay's logarithm, the decay, what the input is multiplied by, and all states."""
    x, gr, gi = s["x"].float(), _sigmoid(s["r"].float()), _sigmoid(s["i"].float())
    la = -DECAY * torch.nn.functional.softplus(s["lam"]) * gr
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    if x.dim() == 2:
        return x, gr, gi, la, a, m, 1.0, a * s["h"] + m * gi * x
    live = 1.0
    if "lengths" in s:
        live = (torch.arange(x.shape[1], device="cuda") < s["lengths"][:, None])[..., None].float()
    through = a * live + (1 - live)  # states pass over the padding
    b = m * gi * x * live
    if "h" in s:
        b[:, 0] += through[:, 0] * s["h"]
    return x, gr, gi, la, through, m, live, _recurrence(through, b)


def _plain_recurrence(s):
    *_, live, h = _rec_parts(s)
    return {"y": (h * live).to(s["x"].dtype), "h_out": h[:, -1].contiguous()}


def _plain_recurrence_step(s):
    h = _rec_parts(s)[-1]
    return {"y": h.to(s["x"].dtype), "h_out": h}


def _plain_recurrence_backward(s):
    x, gr, gi, la, a, m, live, h = _rec_parts(s)
    io = s["x"].dtype
    ahead = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    q = _recurrence(ahead, (s["d_y"].float() * live).flip(1)).flip(1)
    h0 = s["h"][:, None] if "h" in s else torch.zeros_like(h[:, :1])
    before = torch.cat([h0, h[:, :-1]], 1)
    out = {"d_h0": a[:, 0] * q[:, 0]} if "h" in s else {}
    q = q * live
    t = q * la * (a * before - a * a / m * gi * x)
    out["d_x"] = (q * m * gi).to(io)
    out["d_r"] = (t * (1 - gr)).to(io)
    out["d_i"] = (q * m * x * gi * (1 - gi)).to(io)
    out["d_lam"] = t.sum((0, 1)) * _sigmoid(s["lam"]) / torch.nn.functional.softplus(s["lam"])
    return out


_PLAIN = {
    ("rmsnorm", "forward"): _plain_rmsnorm, ("rmsnorm", "e4m3"): _plain_rmsnorm_e4m3,
    ("rmsnorm", "backward"): _plain_rmsnorm_backward, ("dropout", "forward"): _plain_dropout,
    ("dropout", "backward"): _plain_dropout_backward, ("recurrence", "forward"): _plain_recurrence,
    ("recurrence", "step"): _plain_recurrence_step, ("recurrence", "backward"): _plain_recurrence_backward,
}


# ------------------------------------------------------------------ the definitions in 64 bits
def _factors(rng, p, M, C):
    """What dropout multiplies by, the generator written out in unsigned 64-bit numbers on the host."""
    seed, offset = (np.uint64(v & (2 ** 64 - 1)) for v in rng.tolist())
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    per = -(-C // 8)
    count = offset + np.arange(M * per, dtype=np.uint64)
    x = [count & low, count >> half, np.zeros_like(count), np.zeros_like(count)]
    key = [int(seed & low), int(seed >> half)]
    for _ in range(10):
        left, right = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(right >> half) ^ x[1] ^ np.uint64(key[0]), right & low, (left >> half) ^ x[3] ^ np.uint64(key[1]), left & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    numbers = np.empty((M * per, 8), dtype=np.int64)
    for j in range(8):
        numbers[:, j] = (x[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)
    least = int(round(p * 65536))
    keep = numbers.reshape(M, per * 8)[:, :C] >= least
    return torch.from_numpy(keep).cuda().double() * (65536.0 / (65536 - least))


def exact(case, seed):
    s = prepare(case, seed)
    v = {k: t.double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point() and k != "h_out"}
    if case["op"] == "dropout":
        factor = _factors(s["rng"], case["p"], case["M"], case["C"])
        if case["direction"] == "backward":
            return {"d_x": v["d_y"] * factor}
        return {"y": v["x"] * factor + v.get("residual", 0)}
    if case["op"] == "rmsnorm":
        return _define_norm(case, s, v)
    step = case["direction"] == "step"
    if step:  # a sequence of one token
        v |= {k: v[k][:, None] for k in ("x", "r", "i")}
    if case["direction"] != "backward":
        with torch.no_grad():
            y, h = _define_recurrence(s, v)
        return {"y": y[:, 0] if step else y, "h_out": h}
    names = [k for k in ("x", "r", "i", "lam", "h") if k in v]
    leaves = [v[k].requires_grad_() for k in names]
    y, _ = _define_recurrence(s, v)
    return dict(zip(["d_h0" if k == "h" else "d_" + k for k in names], torch.autograd.grad(y, leaves, v["d_y"])))


def _define_norm(case, s, v):
    factor = _factors(s["rng"], case["p"], case["M"], case["D"]) if case["p"] > 0 else 1.0

    def normed(t, w):
        return t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS) * w

    if case["direction"] == "backward":
        t, w = v["x"].requires_grad_(), v["weight"].requires_grad_()
        d_t, d_w = torch.autograd.grad(normed(t, w), (t, w), v["d_y"])
        d_t = d_t + v.get("d_sum", 0)
        return {"d_s": d_t, "d_weight": d_w} | ({"d_x": d_t * factor} if case["p"] > 0 else {})
    total = v["x"] * factor + v.get("residual", 0)
    y = normed(total, v["weight"])
    out = {"sum": total} if "residual" in v else {}
    if case["direction"] == "forward":
        return out | {"y": y}
    y = y.unflatten(-1, (-1, case["group"] or case["D"]))
    scales = y.abs().amax(-1) / 448
    y = (y / scales[..., None]).flatten(-2)
    # the nearest number with three bits behind the leading one, in steps of 2^-9 at least, ties to the even one
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return out | {"y": torch.round(y / unit) * unit, "scales": scales}


def _define_recurrence(s, v):
    """The recurrence token after token."""
    x = v["x"]
    B, N, C = x.shape
    la = -DECAY * torch.nn.functional.softplus(v["lam"], threshold=50.0) * torch.sigmoid(v["r"])
    drive = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(v["i"]) * x
    decay = torch.exp(la)
    h = v["h"] if "h" in v else x.new_zeros(B, C)
    if "lengths" in s:
        inside = torch.arange(N, device="cuda")[:, None] < s["lengths"]  # [N, B]
        decay = torch.where(inside.t()[..., None], decay, 1.0)
        drive = torch.where(inside.t()[..., None], drive, 0.0)
    ys = []
    for a, b in zip(decay.unbind(1), drive.unbind(1)):
        h = a * h + b
        ys.append(h)
    y = torch.stack(ys, 1)
    if "lengths" in s:
        y = torch.where(inside.t()[..., None], y, 0.0)
    return y, h
