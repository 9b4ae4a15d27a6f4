"""The block operators at real lengths, entry by entry against float64 within what fp32 can lose (seq_reference.py): walks of
several turns, segments of many tokens, slow decays."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import seq_reference as R  # noqa: E402
from seq_helpers import Inputs, sliced  # noqa: E402
from seq_plans import CONV_CASES, NORM_CASES, SCAN_CASES, scan_segments  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

EPS = 1e-5
DT = {"bf16": T.TTT_BF16, "fp32": T.TTT_F32}
ids = lambda c: "-".join(str(v) for v in c if not isinstance(v, (dict, list)))  # noqa: E731


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("case", NORM_CASES, ids=ids)
def test_layernorm(case):
    """A row's sums: at most 24 elements in a lane, 6 levels over lanes, 16 waves. A parameter's: a group's turns, at most
    128 groups of a workgroup, and the partial rows, 64 at a time and 6 levels."""
    M, H, D, dtype, cut, at_once = case
    print(f"layernorm M={M} H={H} D={D} {dtype} sliced={cut}", flush=True)
    assert M > 2 * at_once and M % at_once
    i = Inputs(M + D, dtype)
    shape = (M, H, D) if H > 1 else (M, D)
    x, d_y = i.normal(*shape, mean=0.5), i.normal(*shape)
    w, b = i.param(*shape[1:], scale=0.2, mean=1.0), i.param(*shape[1:], scale=0.3)
    x = sliced(x, 1, 8) if cut else x
    rows = T.load_library().ttt_backward_layernorm_workspace(DT[dtype], M, H, D) // (8 * H * D)
    ref = R.layernorm(x, w, b, d_y, EPS, 24 + 6 + 16, M // at_once + 1 + 128 + rows // 64 + 7)
    R.held("y", T.ttt_forward_layernorm(x, w, b, EPS), ref["y"])
    for name, got in zip(("d_x", "d_weight", "d_bias"), T.ttt_backward_layernorm(x, w, d_y, EPS)):
        R.held(name, got, ref[name])


@pytest.mark.parametrize("case", CONV_CASES, ids=ids)
def test_conv1d(case):
    """A parameter's sums: a run of at most 32 tokens, 8 runs of a workgroup, and the partial rows of at least 8 runs of 4
    tokens, 64 at a time and 6 levels."""
    B, N, C, K, dtype, silu, state, lengths = case
    print(f"conv1d B={B} N={N} C={C} K={K} {dtype}", flush=True)
    i = Inputs(N + C, dtype)
    x, d_y, w, b = i.normal(B, N, C), i.normal(B, N, C), i.param(C, K, scale=0.5), i.param(C, scale=0.1)
    s = i.normal(B, K - 1, C) if state else None
    more = dict(silu=silu, state=s, lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    ref = R.conv1d(x, w, b, d_y, rows_depth=32 + 8 + B * (N // 32 + 1) // 64 + 7, **more)
    R.held("y", T.ttt_forward_conv1d(x, w, b, **more), ref["y"])
    for name, got in zip(("d_x", "d_weight", "d_bias", "d_state"), T.ttt_backward_conv1d(x, w, b, d_y, **more)):
        if got is not None:
            R.held(name, got, ref[name])


def _scan_inputs(B, N, C, S, G, dtype, gate=True, lengths=None, sp=True):
    """Half of the states decay by about a thousandth a token, so that start states are there at every segment's end."""
    i = Inputs(N + C + S, dtype)
    s = dict(u=i.normal(B, N, C), delta=i.normal(B, N, C, scale=0.5), Bm=i.normal(B, N, G, S), Cm=i.normal(B, N, G, S),
             D=i.param(C), delta_bias=i.param(C, scale=0.5, mean=-3.0), z=i.normal(B, N, C) if gate else None, h0=i.param(B, C, S))
    fast = 0.5 + torch.arange(S) + torch.rand(C, S, generator=i.gen)
    s["A"] = -torch.where(torch.arange(S) % 2 == 0, 0.02 * fast / S, fast).cuda()
    s["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if not sp:
        s["delta"], s["delta_bias"] = (s["delta"].abs() * 0.1 + 0.01).to(i.io), None
    return dict(s, softplus=sp), i.normal(B, N, C)


@pytest.mark.parametrize("case", SCAN_CASES, ids=ids)
def test_scan_forward(case):
    """(A call without lengths may have fewer segments than the workspace is for, three for four.)"""
    B, N, C, S, G, dtype, opt = case[:7]
    print(f"scan forward B={B} N={N} C={C} S={S} G={G} {dtype} {opt}", flush=True)
    s, _ = _scan_inputs(B, N, C, S, G, dtype, **opt)
    end = torch.full((B, C, S), 7.0, device="cuda")
    y = T.ttt_forward_selective_scan(**s, h_out=end)
    nseg, tokens = scan_segments(B, N, C, S, G, dtype=DT[dtype])
    ref = R.scan(**s, tokens=1 if nseg == 1 else 2 * tokens)
    R.held("y", y, ref["y"])
    R.held("h_out", end, ref["h_out"])


@pytest.mark.parametrize("case", SCAN_CASES, ids=ids)
def test_scan_backward(case):
    """A parameter's sums: a segment's tokens, 8 waves, and the segments, 64 at a time and 6 levels."""
    B, N, C, S, G, dtype, opt = case[:7]
    print(f"scan backward B={B} N={N} C={C} S={S} G={G} {dtype} {opt}", flush=True)
    s, d_y = _scan_inputs(B, N, C, S, G, dtype, **opt)
    names = ("d_u", "d_delta", "d_A", "d_B", "d_C", "d_D", "d_delta_bias", "d_z", "d_h0")
    got = dict(zip(names, T.ttt_backward_selective_scan(**s, d_y=d_y)))
    nseg, tokens = scan_segments(B, N, C, S, G, backward=True, dtype=DT[dtype])
    tokens = min(N, tokens + 8)
    ref = R.scan(**s, d_y=d_y, tokens=tokens, depth=tokens + 8 + B * nseg // 64 + 7)
    for name in names:
        if got[name] is not None:
            R.held(name, got[name], ref[name])
