"""The block operators together, as a sequence block uses them, and what they share: norm, projection, short
convolution with SiLU, projections of the step, B and C, gated scan; a prompt and then single tokens, and the
gradients through all of it. Rows beyond 32-bit offsets, two streams at once.

Bounds: tests/seq_helpers.py. In the chains every stage's output is rounded to the I/O type before the
next; the oracle's chain is given the same rounded values (the library's own outputs), so that each stage
is held to its own bound.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T
from oracle import seq_oracle as O
from seq_helpers import C_CONV, C_NORM, C_SCAN, C_SUM, Inputs, check, f64

EPS = 1e-5
B, N, WIDTH, C, S, G, K, RANK = 2, 70, 48, 80, 16, 1, 4, 8


def _weights(dtype):
    i = Inputs(5, dtype)
    w = {"norm_w": i.param(WIDTH, scale=0.1, mean=1.0), "norm_b": i.param(WIDTH, scale=0.1),
         "w_in": i.normal(WIDTH, 2 * C, scale=WIDTH ** -0.5), "conv_w": i.param(C, K, scale=0.5), "conv_b": i.param(C, scale=0.1),
         "w_proj": i.normal(C, RANK + 2 * G * S, scale=C ** -0.5), "w_step": i.normal(RANK, C, scale=RANK ** -0.5),
         "A": -(torch.arange(S) + 0.5 + torch.rand(C, S, generator=i.gen)).cuda(), "D": i.param(C),
         "dbias": i.param(C, scale=0.5, mean=-3.0)}
    return i, w


def _stages(x, w, conv_state=None, h=None, step=False):
    """One block up to its output projection; every stage's tensors by name. A step updates the states."""
    t = {"x": x, "normed": T.ttt_forward_layernorm(x, w["norm_w"], w["norm_b"], EPS)}
    both = t["normed"] @ w["w_in"]
    t["branch"], t["z"] = both[..., :C], both[..., C:]
    if step:
        t["u"] = T.ttt_step_conv1d(t["branch"], w["conv_w"], w["conv_b"], silu=True, state=conv_state)
    else:
        t["u"] = T.ttt_forward_conv1d(t["branch"], w["conv_w"], w["conv_b"], silu=True, state_out=conv_state)
    proj = t["u"] @ w["w_proj"]
    t["delta"] = proj[..., :RANK] @ w["w_step"]
    t["Bm"] = proj[..., RANK:RANK + G * S].unflatten(-1, (G, S))
    t["Cm"] = proj[..., RANK + G * S:].unflatten(-1, (G, S))
    scan_in = (t["u"], t["delta"], w["A"], t["Bm"], t["Cm"], w["D"], w["dbias"], t["z"])
    if step:
        t["y"] = T.ttt_step_selective_scan(*scan_in, h=h)
    else:
        t["y"] = T.ttt_forward_selective_scan(*scan_in, h_out=h)
    return t


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_block_prompt_then_tokens(dtype):
    i, w = _weights(dtype)
    x = i.normal(B, N + 5, WIDTH)
    conv_state, h = torch.empty(B, K - 1, C, device="cuda", dtype=i.io), torch.empty(B, C, S, device="cuda")
    t = _stages(x[:, :N].contiguous(), w, conv_state, h)
    v = {k: f64(a) for k, a in (t | w).items()}
    check("normed", t["normed"], O.layernorm(v["x"], v["norm_w"], v["norm_b"], EPS), C_NORM)
    ru, rstate = O.conv1d(v["branch"], v["conv_w"], v["conv_b"], True)
    check("u", t["u"], ru, C_CONV)
    check("conv state", conv_state, rstate, 0)
    ry, rh = O.scan(v["u"], v["delta"], v["A"], v["Bm"], v["Cm"], v["D"], v["dbias"], v["z"])
    check("y", t["y"], ry, C_SCAN)
    check("h", h, rh, C_SCAN)
    for n in range(N, N + 5):
        before_conv, before_h = f64(conv_state), f64(h)
        t = _stages(x[:, n], w, conv_state, h, step=True)
        v = {k: f64(a) for k, a in (t | w).items()}
        ru, rstate = O.conv1d(v["branch"][:, None], v["conv_w"], v["conv_b"], True, state=before_conv)
        check(f"u {n}", t["u"], ru[:, 0], C_CONV)
        check("conv state", conv_state, rstate, 0)
        ry, rh = O.scan(*(v[k][:, None] if k not in ("A",) else v[k] for k in ("u", "delta", "A", "Bm", "Cm")), v["D"],
                        v["dbias"], v["z"][:, None], h0=before_h)
        check(f"y {n}", t["y"], ry[:, 0], C_SCAN)
        check("h", h, rh, C_SCAN)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_block_gradients(dtype):
    """The backward passes in the order a training step calls them, the projections' between them by torch."""
    i, w = _weights(dtype)
    x, d_y = i.normal(B, N, WIDTH), i.normal(B, N, C)
    t = _stages(x, w)
    v = {k: f64(a) for k, a in (t | w).items()}
    g = dict(zip(("d_u", "d_delta", "d_A", "d_B", "d_C", "d_D", "d_delta_bias", "d_z"),
                 T.ttt_backward_selective_scan(t["u"], t["delta"], w["A"], t["Bm"], t["Cm"], d_y, w["D"], w["dbias"], t["z"])))
    r = O.scan_backward(v["u"], v["delta"], v["A"], v["Bm"], v["Cm"], f64(d_y), v["D"], v["dbias"], v["z"])
    for k, a in g.items():
        check(k, a, r[k], C_SUM if k in ("d_A", "d_D", "d_delta_bias", "d_B", "d_C") else 4 * C_SCAN)
    d_proj = torch.cat([g["d_delta"] @ w["w_step"].t(), g["d_B"].flatten(-2), g["d_C"].flatten(-2)], -1)
    d_u = g["d_u"] + d_proj @ w["w_proj"].t()
    got = T.ttt_backward_conv1d(t["branch"], w["conv_w"], w["conv_b"], d_u, silu=True)
    for k, a, b, c in zip(("d_branch", "d_conv_w", "d_conv_b"), got,
                          O.conv1d_backward(v["branch"], v["conv_w"], v["conv_b"], True, f64(d_u)), (C_CONV, C_SUM, C_SUM)):
        check(k, a, b, c)
    d_normed = torch.cat([got[0], g["d_z"]], -1) @ w["w_in"].t()
    got = T.ttt_backward_layernorm(x, w["norm_w"], d_normed, EPS)
    for k, a, b, c in zip(("d_x", "d_norm_w", "d_norm_b"), got, O.layernorm_backward(v["x"], v["norm_w"], f64(d_normed), EPS),
                          (C_NORM, C_SUM, C_SUM)):
        check(k, a, b, c)


def test_norm_of_heads_before_a_ttt_layer():
    """Queries and keys normed per head, read out of a fused projection's rows, then the causal layer: the
    layer takes the norm's output as it is, and gives the bits it gives on the same values anywhere."""
    i = Inputs(8, "bf16")
    H, D = 3, 64
    qkv = i.normal(2, 128, 3 * H * D)
    w, b = i.param(H, D, scale=0.1, mean=1.0), i.param(H, D, scale=0.1)
    q, k = (T.ttt_forward_layernorm(qkv[..., j * H * D:(j + 1) * H * D].unflatten(-1, (H, D)), w, b, EPS) for j in (0, 1))
    for j, t in ((0, q), (1, k)):
        check("normed", t, O.layernorm(f64(qkv[..., j * H * D:(j + 1) * H * D].unflatten(-1, (H, D))), f64(w), f64(b), EPS), C_NORM)
    v = qkv[..., 2 * H * D:].unflatten(-1, (H, D)).contiguous()
    w0 = i.param(H, D, D, scale=0.02)
    o = T.ttt_forward_chunked_causal(q * 0.125, k * 0.125, v, w0, 16)
    again = T.ttt_forward_chunked_causal((q * 0.125).clone(), (k * 0.125).clone(), v.clone(), w0, 16)
    assert torch.equal(o, again) and torch.isfinite(o.float()).all()


def test_rows_past_32_bits():
    """Slices whose rows lie 2^30 elements apart (four rows: past 2^31 elements and 2^32 bytes)."""
    i = Inputs(9, "bf16")
    n, c, far = 4, 24, 1 << 30
    hold = torch.empty((n - 1) * far + 4 * c, dtype=torch.bfloat16, device="cuda")

    def spread(t, col):  # t [1, n, w] as a strided view of hold, at column col
        view = hold[col:].as_strided((1, n, t.shape[-1]), (n * far, far, 1))
        view.copy_(t)
        return view

    x = i.normal(1, n, c)
    w, b = i.param(c), i.param(c)
    far_x = spread(x, 0)
    check("layernorm", T.ttt_forward_layernorm(far_x, w, b, EPS), O.layernorm(f64(x), f64(w), f64(b), EPS), C_NORM)
    d_y = i.normal(1, n, c)
    for g, r, cc in zip(T.ttt_backward_layernorm(far_x, w, d_y, EPS), O.layernorm_backward(f64(x), f64(w), f64(d_y), EPS),
                        (C_NORM, C_SUM, C_SUM)):
        check("layernorm backward", g, r, cc)
    taps = i.param(c, 4)
    check("conv1d", T.ttt_forward_conv1d(far_x, taps, b), O.conv1d(f64(x), f64(taps), f64(b), False)[0], C_CONV)
    for g, r, cc in zip(T.ttt_backward_conv1d(far_x, taps, b, d_y), O.conv1d_backward(f64(x), f64(taps), f64(b), False, f64(d_y)),
                        (C_CONV, C_SUM, C_SUM)):
        check("conv1d backward", g, r, cc)
    delta, bm, cm = i.normal(1, n, c, scale=0.5), i.normal(1, n, 8), i.normal(1, n, 8)
    A = -(torch.arange(8) + 1.0).repeat(c, 1).cuda()
    ins = (far_x, spread(delta, c), A, spread(bm, 2 * c).unflatten(-1, (1, 8)), spread(cm, 3 * c).unflatten(-1, (1, 8)))
    ref = (f64(x), f64(delta), f64(A), f64(bm)[:, :, None], f64(cm)[:, :, None])
    check("scan", T.ttt_forward_selective_scan(*ins), O.scan(*ref)[0], C_SCAN)
    r = O.scan_backward(*ref, f64(d_y))
    for name, g in zip(("d_u", "d_delta", "d_A", "d_B", "d_C"), T.ttt_backward_selective_scan(*ins, d_y)):
        check(name, g, r[name], C_SUM)


def test_outputs_past_32_bits():
    """More than 2^32 elements out: the last rows against the oracle. The scan's steps are at least 1 with A =
    -8, so that 16 tokens back nothing of the state is left (exp(-128)) and the oracle starts there."""
    rows, width = (1 << 22) - 3, 1040
    x = torch.empty(1, rows, width, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    i = Inputs(10, "bf16")
    tail = i.normal(1, 40, width)
    x[:, -40:] = tail
    w, b = i.param(width), i.param(width)
    y = T.ttt_forward_layernorm(x, w, b, EPS)
    check("layernorm", y[:, -40:], O.layernorm(f64(tail), f64(w), f64(b), EPS), C_NORM)
    taps = i.param(width, 4)
    T.ttt_forward_conv1d(x, taps, b, y=y)
    check("conv1d", y[:, -37:], O.conv1d(f64(tail), f64(taps), f64(b), False)[0][:, 3:], C_CONV)
    mats = i.normal(1, 40, 16)
    both = torch.zeros(1, rows, 16, dtype=torch.bfloat16, device="cuda")
    both[:, -40:] = mats
    delta = torch.full((1, 1, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    delta = delta.expand(1, rows, width).contiguous()
    A = torch.full((width, 8), -8.0, device="cuda")
    bm, cm = both[..., :8].unflatten(-1, (1, 8)), both[..., 8:].unflatten(-1, (1, 8))
    T.ttt_forward_selective_scan(x, delta, A, bm, cm, y=y)
    ref = O.scan(f64(tail), np.full((1, 40, width), 2.0), f64(A), f64(mats)[:, :, None, :8], f64(mats)[:, :, None, 8:])[0]
    check("scan", y[:, -20:], ref[:, -20:], C_SCAN)


def test_two_streams_at_once():
    """Calls in flight together on two streams, each with the workspace it allocates there."""
    i = Inputs(11, "bf16")
    c, n = 192, 600
    ins = [(i.normal(1, n, c), i.normal(1, n, c, scale=0.5), -(torch.arange(16) + 1.0).repeat(c, 1).cuda(), i.normal(1, n, 1, 16),
            i.normal(1, n, 1, 16)) for _ in range(2)]
    d_y = i.normal(1, n, c)
    want = [(T.ttt_forward_selective_scan(*a), *T.ttt_backward_selective_scan(*a, d_y)[:5]) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for a, s in zip(ins, streams):
            got.append((T.ttt_forward_selective_scan(*a, stream=s), *T.ttt_backward_selective_scan(*a, d_y, stream=s)[:5]))
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(outs, want[k % 2]))
