"""GPU parity of the selective state space scan, forward, backward and single tokens, against the fp64
oracle (bounds: tests/seq_helpers.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T
from oracle import seq_oracle as O
from seq_helpers import C_SCAN, C_SUM, Inputs, check, f64, replays, sliced

NAMES = ("d_u", "d_delta", "d_A", "d_B", "d_C", "d_D", "d_delta_bias", "d_z", "d_h0")


def _inputs(B, N, C, S, G, dtype, gate=True, state=True, lengths=None, cut=False, params=True, sp=True, seed=0):
    """Steps from 0.01 (softplus of about -4.6) up, A in -[0.5, S + 0.5]."""
    i = Inputs(seed, dtype)
    s = {"u": i.normal(B, N, C), "delta": i.normal(B, N, C, scale=0.5), "Bm": i.normal(B, N, G, S),
         "Cm": i.normal(B, N, G, S), "z": i.normal(B, N, C) if gate else None, "d_y": i.normal(B, N, C)}
    s["A"] = -(torch.arange(S) + 0.5 + torch.rand(C, S, generator=i.gen)).cuda()
    s["D"] = i.param(C) if params else None
    s["delta_bias"] = i.param(C, scale=0.5, mean=-3.0) if params else None
    if not sp:
        s["delta"] = (0.01 + 0.3 * torch.rand(B, N, C, generator=i.gen)).to(i.io).cuda()
        s["delta_bias"] = None
    s["h0"] = i.param(B, C, S) if state else None
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths else None
    if lengths:  # padding holds anything
        for j, n in enumerate(lengths):
            for k in ("u", "delta", "Bm", "Cm", "z", "d_y"):
                if s[k] is not None:
                    s[k][j, max(n, 0):] = float("nan") if k != "u" else float("inf")
    if cut:
        for k in ("u", "delta", "Bm", "Cm", "z"):
            if s[k] is not None:
                s[k] = sliced(s[k], 2, 6)
    return s


def _args(s):
    return s["u"], s["delta"], s["A"], s["Bm"], s["Cm"]


def _oracle(s, sp, lengths, backward=False):
    v = {k: f64(s[k]) for k in ("u", "delta", "A", "Bm", "Cm", "D", "z", "h0")}
    v |= {"dbias": f64(s["delta_bias"]), "sp": sp, "lengths": lengths}
    return O.scan_backward(dy=f64(s["d_y"]), **v) if backward else O.scan(**v)


CASES = [  # B, N, C, S, G, dtype, options
    (1, 1, 1, 8, 1, "fp32", {}),
    (2, 1, 64, 16, 1, "bf16", dict(cut=True)),
    (1, 3, 65, 16, 1, "fp32", dict(gate=False)),
    (3, 15, 7, 32, 1, "fp32", dict(lengths=[15, 0, 1])),
    (2, 16, 128, 16, 2, "bf16", dict(state=False)),
    (1, 17, 130, 16, 2, "fp32", dict(cut=True)),
    (2, 33, 24, 64, 3, "fp32", dict(params=False)),
    (1, 64, 96, 8, 1, "bf16", {}),
    (3, 65, 100, 16, 4, "fp32", dict(lengths=[65, 64, 17], cut=True)),
    (2, 129, 70, 16, 1, "bf16", dict(lengths=[129, 100])),
    (1, 200, 80, 32, 5, "bf16", dict(gate=False)),
    (1, 257, 64, 64, 1, "bf16", {}),
    (2, 300, 66, 8, 2, "fp32", dict(sp=False)),
    (4, 301, 36, 16, 1, "fp32", dict(lengths=[301, -3, 900, 250])),
    (1, 1500, 48, 16, 1, "fp32", dict(state=False)),
    (1, 2049, 20, 32, 2, "bf16", dict(cut=True)),
]


@pytest.mark.parametrize("B,N,C,S,G,dtype,opt", CASES, ids=lambda v: str(v))
def test_scan_forward(B, N, C, S, G, dtype, opt):
    print(f"scan forward B={B} N={N} C={C} S={S} G={G} {dtype} {opt}", flush=True)
    s, sp, lengths = _inputs(B, N, C, S, G, dtype, seed=N + C, **opt), opt.get("sp", True), opt.get("lengths")
    end = torch.full((B, C, S), 7.0, device="cuda")
    y = T.ttt_forward_selective_scan(*_args(s), s["D"], s["delta_bias"], s["z"], softplus=sp, h0=s["h0"],
                                     lengths=s["lengths"], h_out=end)
    torch.cuda.synchronize()
    ry, rend = _oracle(s, sp, lengths)
    check("y", y, ry, C_SCAN)
    check("h_out", end, rend, C_SCAN)


@pytest.mark.parametrize("B,N,C,S,G,dtype,opt", CASES, ids=lambda v: str(v))
def test_scan_backward(B, N, C, S, G, dtype, opt):
    print(f"scan backward B={B} N={N} C={C} S={S} G={G} {dtype} {opt}", flush=True)
    s, sp, lengths = _inputs(B, N, C, S, G, dtype, seed=N + C, **opt), opt.get("sp", True), opt.get("lengths")
    got = T.ttt_backward_selective_scan(*_args(s), s["d_y"], s["D"], s["delta_bias"], s["z"], softplus=sp, h0=s["h0"],
                                        lengths=s["lengths"])
    torch.cuda.synchronize()
    ref = _oracle(s, sp, lengths, backward=True)
    for name, g in zip(NAMES, got):
        if g is not None:
            check(name, g, ref[name], C_SUM if name in ("d_A", "d_D", "d_delta_bias", "d_B", "d_C") else 4 * C_SCAN)
    present = {"d_D": "D", "d_delta_bias": "delta_bias", "d_z": "z", "d_h0": "h0"}
    assert all((g is None) == (s.get(present.get(n, "u")) is None) for n, g in zip(NAMES, got))


@pytest.mark.parametrize("B,C,S,G,dtype,gate", [(1, 1, 8, 1, "fp32", True), (5, 66, 16, 2, "bf16", True),
                                                (3, 100, 32, 1, "fp32", False), (7, 33, 64, 3, "bf16", True),
                                                (64, 192, 16, 1, "bf16", True)])
def test_scan_tokens(B, C, S, G, dtype, gate):
    print(f"scan step B={B} C={C} S={S} G={G} {dtype}", flush=True)
    N = 4
    s = _inputs(B, N, C, S, G, dtype, gate=gate, seed=C)
    ry, rend = _oracle(s, True, None)
    h = s["h0"].clone()
    for t in range(N):
        row = [None if s[k] is None else s[k][:, t] for k in ("u", "delta", "Bm", "Cm", "z")]
        out = torch.empty_like(h) if t % 2 else None
        y = T.ttt_step_selective_scan(row[0], row[1], s["A"], row[2], row[3], s["D"], s["delta_bias"], row[4], h=h, h_out=out)
        h = h if out is None else out
        check(f"y {t}", y, ry[:, t], C_SCAN)
    check("h", h, rend, C_SCAN)
    unaligned = torch.empty(B * C * S + 1, device="cuda")[1:].view(B, C, S)
    unaligned.copy_(s["h0"])
    row = [None if s[k] is None else s[k][:, 0] for k in ("u", "delta", "Bm", "Cm", "z")]
    y = T.ttt_step_selective_scan(row[0], row[1], s["A"], row[2], row[3], s["D"], s["delta_bias"], row[4], h=unaligned)
    check("y, state off 16 bytes", y, ry[:, 0], C_SCAN)


def test_scan_continues_from_its_state():
    s = _inputs(2, 700, 72, 16, 2, "fp32", seed=4)
    ry, rend = _oracle(s, True, None)
    h = s["h0"].clone()
    for lo, hi in ((0, 1), (1, 130), (130, 700)):
        part = {k: s[k][:, lo:hi].contiguous() for k in ("u", "delta", "Bm", "Cm", "z")}
        out = torch.empty_like(h)
        y = T.ttt_forward_selective_scan(part["u"], part["delta"], s["A"], part["Bm"], part["Cm"], s["D"], s["delta_bias"],
                                         part["z"], h0=h, h_out=out)
        check(f"y {lo}", y, ry[:, lo:hi], C_SCAN)
        h = out
    check("h", h, rend, C_SCAN)


def test_scan_steps_at_their_ends():
    """softplus far below zero leaves the state as it is (the step underflows), far above it is the sum
    itself and the state is forgotten; at delta -inf nothing turns into NaN."""
    s = _inputs(1, 3, 64, 16, 1, "fp32", gate=False, seed=9)
    s["delta"][0, 0], s["delta"][0, 1], s["delta"][0, 2] = -300.0, 90.0, float("-inf")
    s["delta_bias"] = None
    end = torch.empty(1, 64, 16, device="cuda")
    y = T.ttt_forward_selective_scan(*_args(s), s["D"], h0=s["h0"], h_out=end)
    ry, rend = _oracle(s, True, None)
    check("y", y, ry, C_SCAN)
    check("h_out", end, rend, C_SCAN)
    got = T.ttt_backward_selective_scan(*_args(s), s["d_y"], s["D"], h0=s["h0"])
    for name, g in zip(NAMES, got):
        assert g is None or torch.isfinite(g).all(), name


def test_scan_gradients_against_differences():
    """d_A, d_h0 and d_u of sum(y * d_y) against central differences of the kernel's own forward, in fp32: the
    difference of two sums of 2000 values of about 3, each off by C_SCAN u in the worst case, over 2 h = 0.02,
    and the third-order term; the gradients are about 10."""
    s = _inputs(1, 40, 50, 8, 1, "fp32", seed=21)

    def f():
        y = T.ttt_forward_selective_scan(*_args(s), s["D"], s["delta_bias"], s["z"], h0=s["h0"])
        return float((y.double() * s["d_y"].double()).sum())

    got = dict(zip(NAMES, T.ttt_backward_selective_scan(*_args(s), s["d_y"], s["D"], s["delta_bias"], s["z"], h0=s["h0"])))
    for name, grad, at in (("A", "d_A", (3, 1)), ("A", "d_A", (49, 0)), ("h0", "d_h0", (0, 7, 2)), ("u", "d_u", (0, 11, 13)),
                           ("delta", "d_delta", (0, 20, 5)), ("Bm", "d_B", (0, 2, 0, 4)), ("Cm", "d_C", (0, 39, 0, 7)),
                           ("D", "d_D", (10,)), ("z", "d_z", (0, 8, 8)), ("delta_bias", "d_delta_bias", (30,))):
        keep, step = s[name][at].clone(), 0.01
        s[name][at] = keep + step
        up = f()
        s[name][at] = keep - step
        down = f()
        s[name][at] = keep
        want, have = (up - down) / (2 * step), float(got[grad][at])
        print(f"  {grad}{at}: {have:.5f} against {want:.5f}", flush=True)
        assert abs(want - have) <= 0.01 + 0.01 * abs(want), (name, want, have)


def test_scan_refuses_wrong_tensors():
    s = _inputs(2, 5, 12, 16, 2, "bf16", seed=1)
    ok = dict(u=s["u"], delta=s["delta"], A=s["A"], Bm=s["Bm"], Cm=s["Cm"], D=s["D"])
    z = torch.zeros
    for bad in (dict(delta=s["delta"][:, :4]), dict(A=s["A"].bfloat16()), dict(Bm=s["Bm"][..., :8]), dict(D=s["D"][:6]),
                dict(Cm=s["Cm"].float()), dict(u=s["u"].transpose(0, 1)), dict(u=s["u"][0]), dict(Bm=s["Bm"][:, :, 0]),
                dict(h0=z(2, 12, 8, device="cuda")), dict(lengths=z(2, device="cuda")), dict(z=s["u"].float()),
                dict(y=s["u"].float()), dict(workspace=z(8))):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_selective_scan(**(ok | bad))
    bm = z(2, 5, 2 * 16 + 3, device="cuda", dtype=torch.bfloat16)[..., 1:33].unflatten(-1, (2, 16))
    with pytest.raises(T.TTTError):  # rows of Bm off 4 bytes
        T.ttt_forward_selective_scan(**(ok | dict(Bm=bm)))
    with pytest.raises(T.TTTError):
        T.ttt_forward_selective_scan(**(ok | dict(y=s["delta"])))
    with pytest.raises(T.TTTError):
        T.ttt_forward_selective_scan(**(ok | dict(A=z(12, 4, device="cuda"), Bm=s["Bm"][..., :4].contiguous(),
                                                  Cm=s["Cm"][..., :4].contiguous())))
    with pytest.raises(ValueError):
        T.ttt_backward_selective_scan(*_args(s), s["d_y"], d_z=torch.empty_like(s["u"]))
    with pytest.raises(TypeError):
        T.ttt_step_selective_scan(s["u"][:, 0], s["delta"][:, 0], s["A"], s["Bm"][:, 0], s["Cm"][:, 0], h=None)


def test_scan_replayed_and_on_another_stream():
    s = _inputs(2, 700, 130, 16, 1, "bf16", lengths=[700, 333], cut=True, seed=6)
    io = s["d_y"]
    end, y = torch.empty_like(s["h0"]), torch.empty_like(io)
    mat = torch.empty(2, 700, 1, 16, device="cuda", dtype=io.dtype)
    outs = dict(d_u=torch.empty_like(io), d_delta=torch.empty_like(io), d_A=torch.empty_like(s["A"]), d_B=mat,
                d_C=torch.empty_like(mat), d_D=torch.empty_like(s["D"]), d_delta_bias=torch.empty_like(s["D"]),
                d_z=torch.empty_like(io), d_h0=torch.empty_like(end))
    par = (s["D"], s["delta_bias"], s["z"])
    more = dict(h0=s["h0"], lengths=s["lengths"])

    def call():
        T.ttt_forward_selective_scan(*_args(s), *par, h_out=end, y=y, **more)
        T.ttt_backward_selective_scan(*_args(s), io, *par, **outs, **more)

    replays(call, [y, end, *outs.values()], lambda: T.ttt_forward_selective_scan(*_args(s), *par, **more))
    want = [t.clone() for t in (y, *outs.values())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [T.ttt_forward_selective_scan(*_args(s), *par, stream=side, **more),
           *T.ttt_backward_selective_scan(*_args(s), io, *par, stream=side, **more)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_scan_many_short_sequences():
    """1664 blocks of channels: each runs its 60 tokens in one go."""
    B, N, C, S = 26, 60, 4096, 8
    s = _inputs(B, N, C, S, 1, "bf16", seed=12, lengths=[60 - i for i in range(B)])
    end = torch.empty_like(s["h0"])
    assert T.load_library().ttt_forward_selective_scan_workspace(T.TTT_BF16, B, N, C, S, 1) == 0
    y = T.ttt_forward_selective_scan(*_args(s), s["D"], s["delta_bias"], s["z"], h0=s["h0"], lengths=s["lengths"], h_out=end)
    ry, rend = _oracle(s, True, [60 - i for i in range(B)])
    check("y", y, ry, C_SCAN)
    check("h_out", end, rend, C_SCAN)


@pytest.mark.parametrize("B,N,C,S,G,dtype,opt", [
    (2, 700, 66, 64, 1, "fp32", dict(lengths=[700, 333], cut=True)), (1, 515, 130, 32, 2, "fp32", dict(cut=True)),
    (3, 400, 64, 32, 1, "bf16", dict(lengths=[400, 0, 77])), (2, 611, 40, 64, 4, "bf16", dict(cut=True)),
    (40, 90, 100, 16, 1, "bf16", {}), (2, 1200, 70, 8, 1, "fp32", dict(cut=True, lengths=[1200, 1199]))], ids=lambda v: str(v))
def test_scan_many_segments(B, N, C, S, G, dtype, opt):
    """Wide states and many segments, with rows of B and C that are slices of wider ones."""
    test_scan_forward(B, N, C, S, G, dtype, opt)
    test_scan_backward(B, N, C, S, G, dtype, opt)
