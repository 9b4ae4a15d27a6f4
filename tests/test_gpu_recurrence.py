"""Gated recurrence, forward, single tokens and backward, against float64 within what fp32 can lose, entry by entry
(lm_reference.py)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
from seq_helpers import DT, Inputs, replays, sliced  # noqa: E402
from seq_reference import held  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

CODE = {"bf16": T.TTT_BF16, "fp32": T.TTT_F32}
CASES = [  # B, N, C, dtype, h0, lengths, sliced
    (1, 1, 1, "fp32", False, None, False), (2, 1, 768, "bf16", True, None, False), (1, 2, 3, "bf16", True, None, False),
    (3, 5, 64, "fp32", True, [5, 0, 3], False), (2, 15, 130, "bf16", False, None, True), (2, 16, 128, "bf16", True, [16, 1], False),
    (1, 17, 129, "fp32", False, None, False), (2, 63, 66, "bf16", True, None, True), (2, 64, 256, "fp32", True, [64, 63], False),
    (2, 65, 255, "bf16", True, [1, 65], False), (1, 127, 34, "fp32", True, None, True), (3, 128, 200, "bf16", False, [128, 65, 64], False),
    (1, 129, 128, "fp32", True, None, False), (2, 255, 126, "bf16", True, None, False), (2, 256, 140, "bf16", False, None, True),
    (2, 257, 100, "fp32", True, [257, 256], False), (4, 333, 193, "fp32", True, [0, 333, 100, 1], False),
    (2, 333, 193, "bf16", True, None, True), (1, 511, 2050, "bf16", False, None, False), (1, 1023, 70, "fp32", True, None, False),
    (3, 1999, 1000, "fp32", True, [1999, 777, 1500], False), (2, 2048, 768, "bf16", False, None, True),
    (1, 4097, 300, "bf16", True, None, False), (8, 700, 96, "bf16", True, [700, 0, 1, 64, 65, 256, 257, 699], True),
    # two channels a lane, several groups of tiles, ends in each
    (4, 5000, 386, "bf16", True, [5000, 0, 2049, 4100], True), (4, 5000, 384, "bf16", False, None, False),
    (5, 2500, 258, "fp32", True, [2500, 1024, 1025, 63, 2049], False), (2, 9000, 129, "bf16", True, [9000, 8193], False),
    (1, 16500, 64, "fp32", True, None, False), (1, 10000, 130, "bf16", False, [9001], False), (65, 40, 1, "fp32", True, None, False),
    # the same of odd widths, rows at odd elements
    (4, 1030, 517, "fp32", True, [1030, 64, 0, 1001], True), (6, 700, 771, "bf16", True, None, True),
]
ids = lambda c: "-".join(str(v) for v in c[:5]) + ("-lengths" if c[5] else "") + ("-sliced" if c[6] else "")  # noqa: E731


def _inputs(B, N, C, dtype, h0, lengths, cut, seed=0):
    """Decays from almost none (a = 1 - 1e-5) to almost all at once; padding's rows are NaN."""
    i = Inputs(B + N + C + seed, dtype)
    x, r, g, d_y = i.normal(B, N, C), i.normal(B, N, C, scale=2.0), i.normal(B, N, C, scale=2.0), i.normal(B, N, C)
    lam = i.param(C, scale=4.0, mean=-6.0)
    s = dict(h0=i.param(B, C) if h0 else None)
    if lengths:
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        behind = torch.arange(N, device="cuda")[None] >= s["lengths"][:, None]
        for t in (x, r, g, d_y):
            t[behind] = float("nan")
    if cut:
        extra = 8 if C % 16 == 0 else 4 if C % 2 == 0 else 3
        x, r, g = (sliced(t, 2, extra) for t in (x, r, g))
    return (x, r, g, lam), s, d_y


def _depth(B, N):
    """Additions in d_lam's sums: a thread's tokens, at most 64 of them one after the other, the threads of a workgroup, then the
    partial rows (one for 64 tokens at least, or a sequence), 64 at a time and 6 levels."""
    return 64 + 32 + B * (N // 64 + 1) // 64 + 7


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    B, N, C, dtype = case[:4]
    print(f"recurrence forward {case}", flush=True)
    mats, s, _ = _inputs(*case)
    end, kept = torch.full((B, C), 7.0, device="cuda"), torch.full((B, (N + 63) // 64, C), 7.0, device="cuda")
    y = T.ttt_forward_gated_recurrence(*mats, h_out=end, states=kept, **s)
    ref = R.recurrence(*mats, **s)
    held("y", y, ref["y"])
    held("h_out", end, ref["h_out"])
    held("states", kept, tuple(v[:, ::64] for v in ref["before"]))
    assert torch.equal(T.ttt_forward_gated_recurrence(*mats, **s), y)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case, kept):
    B, N, C, dtype = case[:4]
    print(f"recurrence backward {case} kept={kept}", flush=True)
    mats, s, d_y = _inputs(*case)
    states = None
    if kept:
        states = torch.empty(B, (N + 63) // 64, C, device="cuda")
        T.ttt_forward_gated_recurrence(*mats, states=states, **s)
    got = T.ttt_backward_gated_recurrence(*mats, d_y, states=states, **s)
    ref = R.recurrence(*mats, d_y, depth=_depth(B, N), **s)
    for name, g in zip(("d_x", "d_r", "d_i", "d_lam", "d_h0"), got):
        if g is not None:
            held(name, g, ref[name])
    assert (got[4] is None) == (s["h0"] is None)


GENTLE = [  # cases with whole waves: one and two channels a lane, whole tiles and padding, several groups of tiles
    (1, 64, 64, "fp32", True, None, False), (2, 300, 128, "bf16", True, [300, 129], False), (4, 5000, 384, "bf16", True, None, False),
    (4, 2500, 256, "fp32", True, [2500, 1024, 1025, 63], True), (3, 1999, 1000, "fp32", True, [1999, 777, 1500], False),
    (2, 2048, 768, "bf16", False, None, True), (6, 700, 771, "bf16", True, None, True), (1, 16500, 64, "fp32", False, None, False),
]


def _lam(which, C):
    """Decays whose largest exponent, 8 softplus(lam), is up to 1/4 in every channel, on both sides of it, or up to it but for one
    channel in 64."""
    i = Inputs(C, "fp32")
    lam = i.param(C, scale=1.5, mean=-5.5).clamp(max=-3.46)  # (8 softplus(-3.46) is 0.2475)
    if which == "around":
        lam = -3.45 + i.param(C, scale=0.02)
    elif which == "few":
        lam[C // 2 % 64::64] = 1.0
    return lam


@pytest.mark.parametrize("which", ["gentle", "around", "few"])
@pytest.mark.parametrize("case", GENTLE, ids=ids)
def test_slow_decays(case, which):
    """Waves of slow decays alone, whose tokens are one straight piece of code without exponentials, beside others: forward, and back
    with kept states and without."""
    B, N, C, dtype = case[:4]
    print(f"recurrence {which} {case}", flush=True)
    mats, s, d_y = _inputs(*case)
    mats = (*mats[:3], _lam(which, C))
    steep = 8 * torch.log1p(torch.exp(mats[3].double())) > 0.25
    assert bool(steep.any()) == (which != "gentle") and not bool(steep.all())
    end, kept = torch.full((B, C), 7.0, device="cuda"), torch.full((B, (N + 63) // 64, C), 7.0, device="cuda")
    y = T.ttt_forward_gated_recurrence(*mats, h_out=end, states=kept, **s)
    ref = R.recurrence(*mats, **s)
    held("y", y, ref["y"])
    held("h_out", end, ref["h_out"])
    held("states", kept, tuple(v[:, ::64] for v in ref["before"]))
    ref = R.recurrence(*mats, d_y, depth=_depth(B, N), **s)
    got = T.ttt_backward_gated_recurrence(*mats, d_y, states=kept, **s)
    for name, g in zip(("d_x", "d_r", "d_i", "d_lam", "d_h0"), got):
        if g is not None:
            held(name, g, ref[name])
    for a, b in zip(got, T.ttt_backward_gated_recurrence(*mats, d_y, **s)):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("B,C,dtype,cut", [(1, 1, "fp32", False), (64, 1536, "bf16", True), (3, 77, "bf16", True), (5, 130, "fp32", False),
                                           (200, 33, "fp32", True)])
def test_step(B, C, dtype, cut):
    print(f"recurrence step B={B} C={C} {dtype} sliced={cut}", flush=True)
    mats, s, _ = _inputs(B, 1, C, dtype, True, None, cut)
    ref = R.recurrence(*mats, **s)
    x, r, g = (t[:, 0] for t in mats[:3])
    out, h = torch.empty_like(s["h0"]), s["h0"].clone()
    y = T.ttt_step_gated_recurrence(x, r, g, mats[3], h=h, h_out=out)
    assert torch.equal(h, s["h0"])
    held("y", y, (ref["y"][0][:, 0], ref["y"][1][:, 0]))
    held("h_out", out, ref["h_out"])
    version = h._version
    assert torch.equal(T.ttt_step_gated_recurrence(x, r, g, mats[3], h=h), y)
    assert torch.equal(h, out) and h._version > version


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_prompt_in_pieces_and_single_tokens(dtype):
    """The states of a first piece go into a second one, and those into single tokens: the whole's bounds."""
    mats, s, _ = _inputs(2, 400, 96, dtype, True, None, False)
    cut = lambda a, b: [t[:, a:b].contiguous() for t in mats[:3]] + [mats[3]]  # noqa: E731
    h = torch.empty(2, 96, device="cuda")
    ys = [T.ttt_forward_gated_recurrence(*cut(0, 137), h0=s["h0"], h_out=h)]
    ys.append(T.ttt_forward_gated_recurrence(*cut(137, 390), h0=h.clone(), h_out=h))
    for n in range(390, 400):
        ys.append(T.ttt_step_gated_recurrence(*(t[:, n] for t in mats[:3]), mats[3], h=h)[:, None])
    ref = R.recurrence(*mats, **s)
    held("y", torch.cat(ys, 1), ref["y"])
    held("h_out", h, ref["h_out"])


def test_gates_at_their_ends():
    """Gates shut and wide open, decays of one and of zero (lam far below and above zero): everything is finite, values
    within the bounds where those are, and a channel that never decays keeps its state."""
    B, N = 1, 200
    i = Inputs(3, "fp32")
    lam = torch.tensor([-200.0, -90.0, -30.0, -12.0, 0.0, 30.0, 200.0], device="cuda")
    C = lam.numel()
    x, d_y, h0 = i.normal(B, N, C), i.normal(B, N, C), i.param(B, C)
    r, g = i.normal(B, N, C, scale=30.0), i.normal(B, N, C, scale=30.0)
    r[:, :50], r[:, 50:100] = -200.0, 200.0
    end = torch.empty(B, C, device="cuda")
    y = T.ttt_forward_gated_recurrence(x, r, g, lam, h0=h0, h_out=end)
    grads = T.ttt_backward_gated_recurrence(x, r, g, lam, d_y, h0=h0)
    assert all(torch.isfinite(t).all() for t in (y, end, *grads))
    assert torch.equal(end[:, 0], h0[:, 0]) and not grads[3][0].any()
    ref = R.recurrence(x, r, g, lam, h0=h0)
    rows = [2, 3, 4, 5, 6]  # (softplus of -90 and below is 1e-39 and less)
    held("y", y[:, :, rows], tuple(v[:, :, rows] + (1e-30 if k else 0) for k, v in enumerate(ref["y"])))
    # against differences of the fp64 definition where decays are ordinary
    ref = R.recurrence(x, r, g, lam, d_y, h0=h0, depth=200)
    for name, got in zip(("d_x", "d_r", "d_i", "d_h0"), (*grads[:3], grads[4])):
        v, b = ref[name]
        held(name, got[..., [3, 4]], (v[..., [3, 4]], b[..., [3, 4]] + 1e-30))


def test_what_is_not_finite_stays_in_its_channel_and_sequence():
    mats, s, d_y = _inputs(3, 300, 130, "fp32", True, None, False)
    want, grads = T.ttt_forward_gated_recurrence(*mats, **s), T.ttt_backward_gated_recurrence(*mats, d_y, **s)
    x, r, g, lam = (t.clone() for t in mats)
    x[1, 100, 7], r[1, 200, 64], g[2, 0, 129] = float("nan"), float("nan"), float("inf")
    h0 = s["h0"].clone()
    h0[0, 3] = float("inf")
    y = T.ttt_forward_gated_recurrence(x, r, g, lam, h0=h0)
    clean = torch.ones(3, 130, dtype=torch.bool, device="cuda")
    for b, c in ((1, 7), (1, 64), (2, 129), (0, 3)):
        clean[b, c] = False
    clean = clean[:, None].expand(3, 300, 130)
    assert torch.equal(y[clean], want[clean])
    assert torch.equal(y[1, :100, 7], want[1, :100, 7]) and torch.isnan(y[1, 100:, 7]).all()
    assert torch.equal(y[1, :200, 64], want[1, :200, 64]) and torch.isnan(y[1, 200:, 64]).all()
    got = T.ttt_backward_gated_recurrence(x, r, g, lam, d_y, h0=h0)
    for a, b in zip(got[:3], grads[:3]):
        assert torch.equal(a[clean], b[clean])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_an_infinite_input_is_behind_it_alone(dtype):
    """Within a run of tokens, at a tile's first and last, and so far back that the decays' product is nothing: rows before are the bits of
    the call without it, rows from it on are not finite; infinite gates are gates of 0 and 1."""
    mats, _, d_y = _inputs(1, 3000, 6, dtype, False, None, False)
    want, grads = T.ttt_forward_gated_recurrence(*mats), T.ttt_backward_gated_recurrence(*mats, d_y)
    x, r, g, lam = (t.clone() for t in mats)
    at = (5, 127, 128, 640, 2999, 0)
    for c, n in enumerate(at):
        x[0, n, c] = float("inf") if c % 2 else -float("inf")
    y, got = T.ttt_forward_gated_recurrence(x, r, g, lam), T.ttt_backward_gated_recurrence(x, r, g, lam, d_y)
    for c, n in enumerate(at):
        assert torch.equal(y[0, :n, c], want[0, :n, c]) and not torch.isfinite(y[0, n:, c]).any()
        assert torch.equal(got[0][..., c], grads[0][..., c])  # (x is not in its own gradient)
        assert torch.equal(got[1][0, :n, c], grads[1][0, :n, c]) and torch.equal(got[2][0, :n, c], grads[2][0, :n, c])
    ends = torch.tensor([float("inf"), -float("inf")], device="cuda", dtype=x.dtype).repeat(3)
    r, g = ends.expand(1, 3000, 6).contiguous(), ends.flip(0).expand(1, 3000, 6).contiguous()
    assert torch.isfinite(T.ttt_forward_gated_recurrence(mats[0], r, g, lam)).all()
    assert all(torch.isfinite(t).all() for t in T.ttt_backward_gated_recurrence(mats[0], r, g, lam, d_y)[:4])


def test_an_empty_slots_state_reaches_nothing():
    """A sequence of no tokens with a start state of NaN: its state is handed on, its rows and gradients are zeros, d_lam is clean."""
    mats, s, d_y = _inputs(3, 100, 70, "bf16", True, [100, 0, 50], False)
    want = T.ttt_backward_gated_recurrence(*mats, d_y, **s)
    h0 = s["h0"].clone()
    h0[1] = float("nan")
    end = torch.empty_like(h0)
    y = T.ttt_forward_gated_recurrence(*mats, h0=h0, lengths=s["lengths"], h_out=end)
    assert not y[1].any() and torch.isnan(end[1]).all() and torch.isfinite(end[[0, 2]]).all()
    got = T.ttt_backward_gated_recurrence(*mats, d_y, h0=h0, lengths=s["lengths"])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[4][1].any()


def test_lengths_outside_are_the_nearer_end():
    mats, s, d_y = _inputs(2, 90, 40, "fp32", True, None, False)
    near, far = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([90, 0], [1000, -5]))
    for a, b in zip(T.ttt_backward_gated_recurrence(*mats, d_y, h0=s["h0"], lengths=near),
                    T.ttt_backward_gated_recurrence(*mats, d_y, h0=s["h0"], lengths=far)):
        assert torch.equal(a, b)
    assert torch.equal(T.ttt_forward_gated_recurrence(*mats, h0=s["h0"], lengths=near),
                       T.ttt_forward_gated_recurrence(*mats, h0=s["h0"], lengths=far))


@pytest.mark.parametrize("B,N,C,dtype", [(2, 9000, 129, "bf16"), (4, 1030, 517, "fp32"), (2, 65, 33, "bf16"), (2, 70, 128, "fp32")])
def test_rows_at_any_element_and_what_is_around_them(B, N, C, dtype):
    """Outputs that start one element behind an aligned place: the bits of other calls, and what is before and behind as it was."""
    print(f"recurrence around B={B} N={N} C={C} {dtype}", flush=True)
    mats, s, d_y = _inputs(B, N, C, dtype, True, None, False)
    arounds = []

    def inside(t):
        around = torch.full((t.numel() + 32,), 7.0, dtype=t.dtype, device="cuda")
        arounds.append((around, t.numel()))
        return around[9:9 + t.numel()].view(t.shape)

    want = T.ttt_forward_gated_recurrence(*mats, **s)
    end, kept = inside(s["h0"]), inside(torch.empty(B, (N + 63) // 64, C, device="cuda"))
    assert torch.equal(T.ttt_forward_gated_recurrence(*mats, y=inside(want), h_out=end, states=kept, **s), want)
    want = T.ttt_backward_gated_recurrence(*mats, d_y, **s)
    got = T.ttt_backward_gated_recurrence(*mats, d_y, states=kept, **s,
                                          **{k: inside(t) for k, t in zip(("d_x", "d_r", "d_i", "d_lam", "d_h0"), want)})
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for around, n in arounds:
        assert bool((around[:9] == 7).all()) and bool((around[9 + n:] == 7).all())


@pytest.mark.parametrize("B,N,C,dtype", [(4, 5000, 129, "fp32"), (2, 5000, 257, "fp32"), (3, 6000, 385, "bf16"), (4, 5000, 131, "fp32")])
def test_a_steep_channel_beside_the_last_of_an_odd_width(B, N, C, dtype):
    """One fast decay in the column before the last, slow ones in the last two channels: every call gives the same bits."""
    print(f"recurrence with a steep channel B={B} N={N} C={C} {dtype}", flush=True)
    (x, r, g, lam), s, d_y = _inputs(B, N, C, dtype, True, None, False)
    lam = torch.full_like(lam, -5.0)
    lam[C - 20] = 2.0
    end, kept = torch.empty(B, C, device="cuda"), torch.empty(B, (N + 63) // 64, C, device="cuda")

    def call():
        y = T.ttt_forward_gated_recurrence(x, r, g, lam, h_out=end, states=kept, **s)
        return (y, end.clone(), kept.clone(), *T.ttt_backward_gated_recurrence(x, r, g, lam, d_y, states=kept, **s))

    want = call()
    for name, got, ref in zip(("y", "h_out", "states"), want, (lambda d: (d["y"], d["h_out"], [v[:, ::64] for v in d["before"]]))(
            R.recurrence(x, r, g, lam, **s))):
        held(name, got, tuple(ref))
    ref = R.recurrence(x, r, g, lam, d_y, depth=_depth(B, N), **s)
    for name, got in zip(("d_x", "d_r", "d_i", "d_lam", "d_h0"), want[3:]):
        held(name, got, ref[name])
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("B,N,C,dtype", [(2, 700, 130, "bf16"), (1, 5000, 64, "fp32"), (3, 257, 101, "bf16"), (2, 64, 33, "fp32"),
                                         (1, 1, 8, "bf16")])
def test_workspaces_are_enough_and_not_left(B, N, C, dtype):
    """Workspaces of exactly the size that is asked for, inside a larger buffer that held the largest numbers, NaN or zeros: the
    same results, and the bytes around as they were."""
    print(f"workspaces B={B} N={N} C={C} {dtype}", flush=True)
    lib = T.load_library()
    mats, s, d_y = _inputs(B, N, C, dtype, True, None, False)
    kept = torch.empty(B, (N + 63) // 64, C, device="cuda")
    T.ttt_forward_gated_recurrence(*mats, states=kept, **s)
    end = torch.empty(B, C, device="cuda")
    for need, call in (
            (lib.ttt_forward_gated_recurrence_workspace(CODE[dtype], B, N, C),
             lambda **k: (T.ttt_forward_gated_recurrence(*mats, h_out=end, **s, **k), end.clone())),
            (lib.ttt_backward_gated_recurrence_workspace(CODE[dtype], B, N, C, 0), lambda **k: T.ttt_backward_gated_recurrence(*mats, d_y, **s, **k)),
            (lib.ttt_backward_gated_recurrence_workspace(CODE[dtype], B, N, C, 1),
             lambda **k: T.ttt_backward_gated_recurrence(*mats, d_y, states=kept, **s, **k))):
        want = call()
        for fill in (0x5A, 0x00, 0xFF):
            around = torch.full((need + 8192,), fill, dtype=torch.uint8, device="cuda")
            got = call(workspace=around[4096:4096 + need] if need else None)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert bool((around[:4096] == fill).all()) and bool((around[4096 + need:] == fill).all())
            if need:
                with pytest.raises(T.TTTError):
                    call(workspace=around[4096:4096 + need - 256])


def test_refusals():
    mats, s, d_y = _inputs(2, 90, 40, "fp32", True, None, False)
    x, r, g, lam = mats
    for bad in (dict(x=x.half()), dict(r=r[:, :50]), dict(i=g.bfloat16()), dict(lam=lam[:5]), dict(lam=lam.double()),
                dict(h0=torch.zeros(2, 41, device="cuda")), dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(states=torch.zeros(2, 1, 40, device="cuda")), dict(x=x.transpose(0, 1)), dict(y=x[:1])):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_gated_recurrence(**(dict(x=x, r=r, i=g, lam=lam) | bad))
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(y=x), dict(h_out=s["h0"], h0=s["h0"])):
        with pytest.raises(T.TTTError):
            T.ttt_forward_gated_recurrence(**(dict(x=x, r=r, i=g, lam=lam) | bad))
    for bad in (dict(d_h0=torch.zeros(2, 40, device="cuda")), dict(d_y=d_y[:1]), dict(states=torch.zeros(2, 3, 40, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_backward_gated_recurrence(**(dict(x=x, r=r, i=g, lam=lam, d_y=d_y) | bad))
    with pytest.raises(T.TTTError):
        T.ttt_backward_gated_recurrence(x, r, g, lam, d_y, d_x=d_y)
    with pytest.raises((ValueError, T.TTTError)):
        T.ttt_step_gated_recurrence(x[:, 0], r[:, 0], g[:, 0], lam, h=torch.zeros(1, 40, device="cuda"))


def test_replayed_and_two_at_once():
    """Graphs with workspaces of their own give the eager bits again and again; so do calls on two streams at once."""
    mats, s, d_y = _inputs(2, 1500, 300, "bf16", True, [1500, 900], False)
    y, end = torch.empty_like(d_y), torch.empty(2, 300, device="cuda")
    kept = torch.empty(2, 24, 300, device="cuda")
    grads = [torch.empty_like(d_y) for _ in range(3)] + [torch.empty_like(mats[3]), torch.empty_like(end)]

    def call():
        T.ttt_forward_gated_recurrence(*mats, h_out=end, states=kept, y=y, **s)
        T.ttt_backward_gated_recurrence(*mats, d_y, states=kept, d_x=grads[0], d_r=grads[1], d_i=grads[2], d_lam=grads[3],
                                        d_h0=grads[4], **s)

    outs = [y, end, kept, *grads]
    replays(call, outs, lambda: T.ttt_forward_gated_recurrence(*mats))
    want = [t.clone() for t in outs]
    without = T.ttt_backward_gated_recurrence(*mats, d_y, **s)
    assert all(torch.equal(a, b) for a, b in zip(without, want[3:]))  # (the states are the same, kept or not)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for k in range(12):
        st = streams[k % 3]
        got.append((T.ttt_forward_gated_recurrence(*mats, **s, stream=st),
                    *T.ttt_backward_gated_recurrence(*mats, d_y, **s, stream=st)))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and all(torch.equal(a, b) for a, b in zip(g[1:], want[3:]))


def test_offsets_past_32_bits():
    """Rows whose stride takes them past 2^32 elements: the last sequence's results are those of a call on it alone."""
    B, N, C, wide = 3, 40000, 8, 40000
    rows = torch.zeros(B * N, wide, device="cuda", dtype=torch.bfloat16)  # 9.6 GB, 4.8e9 elements
    i = Inputs(2, "bf16")
    x, r, g = (rows[:, 100 * k:100 * k + C].view(B, N, C) for k in (1, 2, 3))
    for t in (x, r, g):
        t.copy_(i.normal(B, N, C))
    lam, d_y = i.param(C, mean=-5.0), i.normal(B, N, C)
    y, grads = T.ttt_forward_gated_recurrence(x, r, g, lam), T.ttt_backward_gated_recurrence(x, r, g, lam, d_y)
    last = [t[2:].contiguous() for t in (x, r, g)]
    assert torch.equal(y[2:], T.ttt_forward_gated_recurrence(*last, lam))
    for a, b in zip(grads[:3], T.ttt_backward_gated_recurrence(*last, lam, d_y[2:].contiguous())[:3]):
        assert torch.equal(a[2:], b)
