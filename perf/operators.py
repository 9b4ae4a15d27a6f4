"""What is measured of the operators around a TTT layer: layer norm, the short causal convolution and
the selective state space scan, each in its directions.

`own` chooses between the operators' plain forms (elementary torch operations in 32 bits, rounded
once at the end) and the library's entry points; both take what `prepare` gives. `exact` computes
the same outputs in 64 bits from the operators' definitions, the gradients by differentiation.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ the cases
def _ln(name, direction, tokens, H, D, dtype, sliced=False):
    return {"name": name, "op": "layernorm", "direction": direction, "tokens": tokens, "H": H, "D": D, "dtype": dtype,
            "sliced": sliced}


def _conv(name, direction, B, N, C, K, dtype, state=False, ragged=False):
    return {"name": name, "op": "conv1d", "direction": direction, "B": B, "N": N, "C": C, "K": K, "dtype": dtype,
            "state": state, "ragged": ragged}


def _scan(name, direction, B, N, C, S, G, dtype, gate=True, state=False, ragged=False):
    return {"name": name, "op": "scan", "direction": direction, "B": B, "N": N, "C": C, "S": S, "G": G,
            "dtype": dtype, "gate": gate, "state": state, "ragged": ragged}


def listed():
    return [
        # one new token of each of 16 sequences at the language layers' width (12 heads x 64): latency
        _ln("layernorm_fwd_tokens", "forward", 16, 1, 768, "bf16"),
        # the queries of the 4 x 8192-token language layer normed per head, read out of the fused
        # q, k, v projection's rows
        _ln("layernorm_fwd_heads", "forward", 4 * 8192, 12, 64, "bf16", sliced=True),
        # a training step's norm over 64 images of 14 x 14 tokens, width 6 x 64
        _ln("layernorm_bwd_images", "backward", 64 * 196, 1, 384, "bf16"),
        # fp32 training at an odd width and token count: no vector access fits its rows
        _ln("layernorm_bwd_odd", "backward", 1537, 1, 1001, "fp32"),
        # the convolution before a causal layer, two prompts of 16384 tokens that continue earlier ones
        _conv("conv1d_fwd_prompt", "forward", 2, 16384, 768, 4, "bf16", state=True),
        # its training step at 4 x 8192 tokens
        _conv("conv1d_bwd_train", "backward", 4, 8192, 768, 4, "bf16"),
        # one new token for each of 64 sequences
        _conv("conv1d_step", "step", 64, 1, 768, 4, "bf16"),
        # the scan over prompts of the language layer's shape, gated, with the end state kept
        _scan("scan_fwd_prompt", "forward", 4, 8192, 768, 16, 1, "bf16"),
        # a padded fp32 batch of unequal prompts that continue earlier ones, two groups, wide state
        _scan("scan_fwd_ragged", "forward", 3, 1999, 1000, 32, 2, "fp32", state=True, ragged=True),
        # a training step of the scan, gated
        _scan("scan_bwd_train", "backward", 2, 4096, 768, 16, 1, "bf16"),
        # a small fp32 training step at odd sizes, without a gate
        _scan("scan_bwd_odd", "backward", 2, 333, 193, 8, 1, "fp32", gate=False, state=True),
        # one new token for each of 64 sequences
        _scan("scan_step", "step", 64, 1, 1536, 16, 1, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = [work(c) for c in listed()]
    most_bytes, most_flops = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        op = rng.choice(["layernorm", "conv1d", "scan", "scan"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if op == "layernorm":
            H = rng.choice([1, 1, 2, 3, 6, 12])
            D = _log_int(rng, 33, 4096) if H == 1 else rng.choice([16, 32, 64, 128])
            c = _ln("", rng.choice(["forward", "backward"]), _log_int(rng, 1, 40000), H, D, dtype, rng.random() < 0.3)
        else:
            direction = rng.choice(["forward", "backward", "step"])
            C = _log_int(rng, 17, 2048)
            C = C if rng.random() < 0.4 else (C + 15) // 16 * 16
            B = _log_int(rng, 1, 256) if direction == "step" else _log_int(rng, 1, 8)
            N = 1 if direction == "step" else _log_int(rng, 1, 16384)
            state = direction == "step" or rng.random() < 0.5
            ragged = direction != "step" and rng.random() < 0.4
            if op == "conv1d":
                c = _conv("", direction, B, N, C, rng.choice([2, 3, 4]), dtype, state, ragged)
            else:
                G = rng.choice([g for g in (1, 1, 1, 2, 4) if C % g == 0])
                S = rng.choice([8, 16, 16, 32, 64])
                c = _scan("", direction, B, N, C, S, G, dtype, rng.random() < 0.6, state, ragged)
        del c["name"]
        w = work(c)
        cost = 3 if c["direction"] == "backward" else 1  # the backward's intermediates are more
        if w["bytes"] <= most_bytes and cost * w["flops"] <= most_flops:
            return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layernorm":
        rows, width = case["tokens"], case["H"] * case["D"]
        if case["direction"] == "forward":
            return {"bytes": 2 * rows * width * e + 8 * width, "flops": 8 * rows * width}
        return {"bytes": 3 * rows * width * e + 12 * width, "flops": 16 * rows * width}
    B, N, C = case["B"], case["N"], case["C"]
    if case["op"] == "conv1d":
        K = case["K"]
        held = 2 * B * (K - 1) * C * e if case["state"] or case["direction"] == "step" else B * (K - 1) * C * e
        if case["direction"] == "backward":
            held = held if case["state"] else 0
            return {"bytes": 3 * B * N * C * e + held + 8 * (K + 1) * C, "flops": (6 * K + 8) * B * N * C}
        return {"bytes": 2 * B * N * C * e + held + 4 * (K + 1) * C, "flops": (2 * K + 5) * B * N * C}
    S, G, gate = case["S"], case["G"], int(case["gate"])
    params, state = 4 * C * (S + 2), 4 * B * C * S
    if case["direction"] == "backward":
        rows = (5 + 2 * gate) * B * N * C * e + 4 * B * N * G * S * e
        return {"bytes": rows + 2 * params + (2 * state if case["state"] else 0), "flops": (22 * S + 30) * B * N * C}
    rows = (3 + gate) * B * N * C * e + 2 * B * N * G * S * e
    held = 2 if case["state"] or case["direction"] == "step" else 1
    return {"bytes": rows + params + held * state, "flops": (7 * S + 15) * B * N * C}


# ---------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale + mean).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, device="cuda", generator=gen) * (hi - lo) + lo

    s = {"case": dict(case)}
    if case["op"] == "layernorm":
        M, H, D = case["tokens"], case["H"], case["D"]
        # activations of a residual stream: some mean, channels of unequal size
        size = torch.exp(normal(H * D, scale=0.5))
        x = (normal(M, H * D) * size + normal(H * D, scale=0.3)).to(dt)
        if case["sliced"]:
            rows = torch.zeros(M, 3 * H * D, device="cuda", dtype=dt)
            rows[:, :H * D] = x
            x = rows[:, :H * D]
        s["x"] = x.view(M, H, D) if H > 1 else x
        shape = (H, D) if H > 1 else (D,)
        s["weight"] = normal(*shape, scale=0.2, mean=1.0)
        s["bias"] = normal(*shape, scale=0.1)
        if case["direction"] == "backward":
            s["d_y"] = normal(*s["x"].shape, dtype=dt)
        return s
    B, N, C, step = case["B"], case["N"], case["C"], case["direction"] == "step"
    if case["ragged"]:
        lengths = torch.randint(0, N + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
        lengths[0] = N  # a batch is padded to its longest sequence
        s["lengths"] = lengths
    lead = (B,) if step else (B, N)
    both = normal(*lead, 2 * C, dtype=dt)  # what the layer's input projection gives: the branch and its gate
    if case["op"] == "conv1d":
        K = case["K"]
        s["x"] = both[..., :C]
        s["weight"] = normal(C, K, scale=1 / math.sqrt(K))
        s["bias"] = normal(C, scale=0.1)
        if case["state"] or step:
            s["state"] = normal(B, K - 1, C, dtype=dt)
        if step:
            s["state_out"] = torch.empty_like(s["state"])
        elif case["direction"] == "backward":
            s["d_y"] = normal(B, N, C, dtype=dt)
        else:
            s["state_out"] = torch.empty(B, K - 1, C, device="cuda", dtype=dt)
        return s
    S, G = case["S"], case["G"]
    rank = (C // 16 + 3) // 4 * 4  # the low-rank step's columns in the same projection's rows
    proj = normal(*lead, rank + 2 * G * S, dtype=dt)
    s["u"] = torch.nn.functional.silu(normal(*lead, C)).to(dt)
    s["delta"] = normal(*lead, C, scale=0.5, dtype=dt)
    s["A"] = -torch.arange(1, S + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(C, S, scale=0.2))
    s["Bm"] = proj[..., rank:rank + G * S].unflatten(-1, (G, S))
    s["Cm"] = proj[..., rank + G * S:].unflatten(-1, (G, S))
    s["D"] = normal(C, scale=0.1, mean=1.0)
    dt0 = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C))
    s["delta_bias"] = torch.log(torch.expm1(dt0))  # softplus(delta_bias) lies in [0.001, 0.1]
    if case["gate"]:
        s["z"] = both[..., C:]
    if case["state"] or step:
        s["h"] = normal(B, C, S, scale=0.3)
    if case["direction"] == "backward":
        s["d_y"] = normal(B, N, C, dtype=dt)
    else:
        s["h_out"] = torch.empty(B, C, S, device="cuda")
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    return _PLAIN[case["op"], case["direction"]](state)


# -------------------------------------------------------------------------- the library's calls
def _own(s):
    import test_sequence_layers_amd as T

    op, direction = s["case"]["op"], s["case"]["direction"]
    if op == "layernorm":
        if direction == "forward":
            return {"y": T.ttt_forward_layernorm(s["x"], s["weight"], s["bias"], EPS)}
        return dict(zip(("d_x", "d_weight", "d_bias"), T.ttt_backward_layernorm(s["x"], s["weight"], s["d_y"], EPS)))
    if op == "conv1d":
        if direction == "step":
            y = T.ttt_step_conv1d(s["x"], s["weight"], s["bias"], silu=True, state=s["state"], state_out=s["state_out"])
            return {"y": y, "state_out": s["state_out"]}
        more = {"silu": True, "state": s.get("state"), "lengths": s.get("lengths")}
        if direction == "forward":
            y = T.ttt_forward_conv1d(s["x"], s["weight"], s["bias"], state_out=s["state_out"], **more)
            return {"y": y, "state_out": s["state_out"]}
        got = dict(zip(("d_x", "d_weight", "d_bias", "d_state"),
                       T.ttt_backward_conv1d(s["x"], s["weight"], s["bias"], s["d_y"], **more)))
        return {k: v for k, v in got.items() if v is not None}
    mats = (s["u"], s["delta"], s["A"], s["Bm"], s["Cm"])
    rest = (s["D"], s["delta_bias"], s.get("z"))
    if direction == "step":
        y = T.ttt_step_selective_scan(*mats, *rest, h=s["h"], h_out=s["h_out"])
        return {"y": y, "h_out": s["h_out"]}
    more = {"h0": s.get("h"), "lengths": s.get("lengths")}
    if direction == "forward":
        y = T.ttt_forward_selective_scan(*mats, *rest, h_out=s["h_out"], **more)
        return {"y": y, "h_out": s["h_out"]}
    names = ("d_u", "d_delta", "d_A", "d_B", "d_C", "d_D", "d_delta_bias", "d_z", "d_h0")
    got = dict(zip(names, T.ttt_backward_selective_scan(*mats, s["d_y"], *rest, **more)))
    return {k: v for k, v in got.items() if v is not None}


# ------------------------------------------------------------------------------- the plain forms
def _normed(s):
    x = s["x"].float()
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def _plain_layernorm(s):
    xhat, _ = _normed(s)
    return {"y": (xhat * s["weight"] + s["bias"]).to(s["x"].dtype)}


def _plain_layernorm_backward(s):
    xhat, rstd = _normed(s)
    dy = s["d_y"].float()
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return {"d_x": dx.to(s["x"].dtype), "d_weight": (dy * xhat).sum(0), "d_bias": dy.sum(0)}


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _live(s, N):
    """1 for a sequence's own tokens, 0 for the padding behind them: [B, N, 1]."""
    if "lengths" not in s:
        return 1.0
    return (torch.arange(N, device="cuda") < s["lengths"][:, None])[..., None].float()


def _windows(s, x):
    """[B, N, C, K]: every token's last K inputs, the state's before the first token; and the padded inputs."""
    K = s["weight"].shape[1]
    before = s["state"].float() if "state" in s else x.new_zeros(x.shape[0], K - 1, x.shape[2])
    padded = torch.cat([before, x], 1)
    return padded.unfold(1, K, 1), padded


def _plain_conv1d(s):
    x = s["x"].float()
    B, N, C = x.shape
    win, padded = _windows(s, x)
    pre = (win * s["weight"]).sum(-1) + s["bias"]
    y = pre * _sigmoid(pre) * _live(s, N)
    last = s["lengths"].long() if "lengths" in s else torch.full((B,), N, device="cuda")
    at = last[:, None] + torch.arange(padded.shape[1] - N, device="cuda")
    held = torch.gather(padded, 1, at[..., None].expand(-1, -1, C))
    return {"y": y.to(s["x"].dtype), "state_out": held.to(s["x"].dtype)}


def _plain_conv1d_step(s):
    x, before = s["x"].float(), s["state"].float()
    win = torch.cat([before, x[:, None]], 1)
    pre = (win * s["weight"].t()).sum(1) + s["bias"]
    return {"y": (pre * _sigmoid(pre)).to(s["x"].dtype), "state_out": win[:, 1:].to(s["x"].dtype)}


def _plain_conv1d_backward(s):
    x, w = s["x"].float(), s["weight"]
    N, K = x.shape[1], w.shape[1]
    win, _ = _windows(s, x)
    pre = (win * w).sum(-1) + s["bias"]
    sig = _sigmoid(pre)
    dpre = s["d_y"].float() * _live(s, N) * sig * (1 + pre * (1 - sig))
    ahead = torch.nn.functional.pad(dpre, (0, 0, K - 1, K - 1)).unfold(1, K, 1)  # [B, N + K - 1, C, K]
    d_padded = (ahead * w.flip(1)).sum(-1).to(s["x"].dtype)
    out = {"d_x": d_padded[:, K - 1:], "d_weight": (dpre[..., None] * win).sum((0, 1)), "d_bias": dpre.sum((0, 1))}
    if "state" in s:
        out["d_state"] = d_padded[:, :K - 1]
    return out


def _recurrence(a, b):
    """h[t] = a[t] h[t - 1] + b[t] along dim 1 for all t at once: pairs of steps are joined, then pairs of pairs."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _per_channel(m, C):
    """[..., G, S] -> [..., C, S] in 32 bits: channel c takes group c // (C / G)'s row."""
    return m.float().repeat_interleave(C // m.shape[-2], -2)


def _scan_parts(s):
    u = s["u"].float()
    N, C = u.shape[1], u.shape[2]
    live = _live(s, N)
    raw = s["delta"].float() + s["delta_bias"]
    dt = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20)))) * live  # a padded token's step is none
    a = torch.exp(dt[..., None] * s["A"])
    Bc, Cc = _per_channel(s["Bm"], C), _per_channel(s["Cm"], C)
    b = (dt * u)[..., None] * Bc
    if "h" in s:
        b[:, 0] += a[:, 0] * s["h"]
    return u, raw, dt, live, a, Bc, Cc, _recurrence(a, b)


def _plain_scan(s):
    u, _, _, live, _, _, Cc, h = _scan_parts(s)
    y = ((h * Cc).sum(-1) + s["D"] * u) * live
    if "z" in s:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return {"y": y.to(s["u"].dtype), "h_out": h[:, -1].contiguous()}


def _plain_scan_step(s):
    u, C = s["u"].float(), s["u"].shape[1]
    raw = s["delta"].float() + s["delta_bias"]
    dt = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20))))
    h = torch.exp(dt[..., None] * s["A"]) * s["h"] + (dt * u)[..., None] * _per_channel(s["Bm"], C)
    y = (h * _per_channel(s["Cm"], C)).sum(-1) + s["D"] * u
    if "z" in s:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return {"y": y.to(s["u"].dtype), "h_out": h}


def _plain_scan_backward(s):
    u, raw, dt, live, a, Bc, Cc, h = _scan_parts(s)
    B, N, C = u.shape
    S, G, io = s["A"].shape[1], s["Bm"].shape[2], s["u"].dtype
    dy = s["d_y"].float() * live
    out = {}
    if "z" in s:
        z = s["z"].float()
        sig = _sigmoid(z)
        out["d_z"] = (dy * ((h * Cc).sum(-1) + s["D"] * u) * sig * (1 + z * (1 - sig))).to(io)
        dy = dy * z * sig
    d_C = (dy[..., None] * h).view(B, N, G, C // G, S).sum(3).to(io)
    h0 = s["h"] if "h" in s else torch.zeros_like(h[:, 0])
    ah = torch.cat([h0[:, None], h[:, :-1]], 1).mul_(a)  # a[t] h[t - 1]
    del h
    back = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    a0 = a[:, 0].clone()
    del a
    g = _recurrence(back, (dy[..., None] * Cc).flip(1)).flip(1)
    del back, Cc
    d_u = (g * Bc).sum(-1)
    d_dt = d_u * u + (g * ah * s["A"]).sum(-1)
    d_u = d_u * dt + s["D"] * dy
    d_raw = d_dt * _sigmoid(raw) * live
    d_B = (g * (dt * u)[..., None]).view(B, N, G, C // G, S).sum(3).to(io)
    if "h" in s:
        out["d_h0"] = a0 * g[:, 0]
    d_A = (g.mul_(ah) * dt[..., None]).sum((0, 1))
    return out | {"d_u": d_u.to(io), "d_delta": d_raw.to(io), "d_A": d_A, "d_B": d_B, "d_C": d_C,
                  "d_D": (dy * u).sum((0, 1)), "d_delta_bias": d_raw.sum((0, 1))}


_PLAIN = {
    ("layernorm", "forward"): _plain_layernorm, ("layernorm", "backward"): _plain_layernorm_backward,
    ("conv1d", "forward"): _plain_conv1d, ("conv1d", "step"): _plain_conv1d_step,
    ("conv1d", "backward"): _plain_conv1d_backward, ("scan", "forward"): _plain_scan,
    ("scan", "step"): _plain_scan_step, ("scan", "backward"): _plain_scan_backward,
}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    step = case["direction"] == "step"
    ins = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and not k.endswith("_out")}
    if step:  # a sequence of one token
        ins |= {k: ins[k][:, None] for k in ("x", "u", "delta", "Bm", "Cm", "z") if k in ins}
    if case["direction"] != "backward":
        with torch.no_grad():
            out = _define(case, s, ins)
        return {k: v[:, 0] if step and k == "y" else v for k, v in out.items()}
    d_y = ins.pop("d_y")
    if "bias" in ins and case["op"] == "layernorm":
        names = ["x", "weight", "bias"]
    else:
        names = [k for k in ("x", "weight", "bias", "state", "u", "delta", "A", "Bm", "Cm", "D", "delta_bias", "z", "h")
                 if k in ins]
    leaves = [ins[k].detach().requires_grad_() for k in names]
    y = _define(case, s, ins | dict(zip(names, leaves)))["y"]
    called = {"Bm": "d_B", "Cm": "d_C", "h": "d_h0"}
    return dict(zip([called.get(k, "d_" + k) for k in names], torch.autograd.grad(y, leaves, d_y)))


def _define(case, s, v):
    """The operator's outputs, each written out as it is defined, token after token."""
    if case["op"] == "layernorm":
        x = v["x"]
        var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
        return {"y": (x - mean) / torch.sqrt(var + EPS) * v["weight"] + v["bias"]}
    first = v["x"] if case["op"] == "conv1d" else v["u"]
    B, N, C = first.shape
    lengths = s["lengths"] if "lengths" in s else torch.full((B,), N, device="cuda")
    if case["op"] == "conv1d":
        K = case["K"]
        held = v["state"] if "state" in v else first.new_zeros(B, K - 1, C)
        line = torch.cat([held, first], 1)
        pre = v["bias"] + sum(v["weight"][:, k] * line[:, k:k + N] for k in range(K))
        y = torch.nn.functional.silu(pre)
        y = y * (torch.arange(N, device="cuda")[None, :, None] < lengths[:, None, None])
        ends = torch.stack([line[b, n:n + K - 1] for b, n in enumerate(lengths.tolist())])
        return {"y": y, "state_out": ends}
    S, G = case["S"], case["G"]
    h = v["h"] if "h" in v else first.new_zeros(B, C, S)
    h = h.reshape(B, G, C // G, S)
    A = v["A"].view(G, C // G, S)
    dt = torch.nn.functional.softplus(v["delta"] + v["delta_bias"], threshold=50.0).view(B, N, G, C // G, 1)
    drive = dt * v["u"].view(B, N, G, C // G, 1)
    runs = torch.arange(N, device="cuda")[:, None] < lengths  # [N, B]
    runs = runs.view(N, B, 1, 1, 1)
    ragged = "lengths" in s
    ys = []
    for dt_t, drive_t, B_t, C_t, on in zip(dt.unbind(1), drive.unbind(1), v["Bm"].unsqueeze(3).unbind(1),
                                           v["Cm"].unsqueeze(-1).unbind(1), runs.unbind(0)):
        new = torch.exp(dt_t * A) * h + drive_t * B_t
        h = torch.where(on, new, h) if ragged else new
        ys.append(torch.matmul(h, C_t))
    y = torch.stack(ys, 1).view(B, N, C) + v["D"] * v["u"]
    if "z" in v:
        y = y * torch.nn.functional.silu(v["z"])
    if ragged:
        y = y * runs.view(N, B).t()[..., None]
    return {"y": y, "h_out": h.reshape(B, C, S)}
