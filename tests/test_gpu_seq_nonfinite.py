"""The block operators where states or inputs hold infinities or NaN that the formulas do not reach: a sequence of
no tokens, the tokens behind a sequence's end, decays past fp32's range."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T
from seq_helpers import DT, Inputs

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("N,C,K,dtype,silu", [(9, 64, 4, "bf16", True), (70, 33, 3, "fp32", False), (300, 40, 2, "bf16", False)])
def test_conv1d_gradients_of_an_empty_sequence(N, C, K, dtype, silu):
    """Its state is in no product: whatever it holds, every gradient is that of a state of zeros."""
    i = Inputs(N, dtype)
    x, d_y, state = i.normal(3, N, C), i.normal(3, N, C), i.normal(3, K - 1, C)
    w, b = i.param(C, K), i.param(C)
    lengths = torch.tensor([N, 0, 1], dtype=torch.int32, device="cuda")
    state[1] = 0.0
    want = T.ttt_backward_conv1d(x, w, b, d_y, silu=silu, state=state, lengths=lengths)
    for value in (NAN, INF):
        state[1] = value
        got = T.ttt_backward_conv1d(x, w, b, d_y, silu=silu, state=state, lengths=lengths)
        for name, g, r in zip(("d_x", "d_weight", "d_bias", "d_state"), got, want):
            assert torch.isfinite(r).all() and torch.equal(g, r), (name, value)


@pytest.mark.parametrize("N,n,K,dtype", [(9, 9, 4, "fp32"), (9, 6, 3, "bf16"), (100, 64, 4, "bf16"), (64, 64, 2, "fp32")])
def test_conv1d_gradients_behind_an_infinite_last_input(N, n, K, dtype):
    """The last input meets the last tap alone: d_weight of the others has no part of it."""
    i = Inputs(N + K, dtype)
    x, d_y, w = i.normal(1, N, 40), i.normal(1, N, 40), i.param(40, K)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = T.ttt_backward_conv1d(x, w, None, d_y, lengths=lengths)
    x[0, n - 1] = INF
    got = T.ttt_backward_conv1d(x, w, None, d_y, lengths=lengths)
    assert torch.equal(got[1][:, :K - 1], want[1][:, :K - 1]) and not torch.isfinite(got[1][:, K - 1]).any()
    assert torch.equal(got[0], want[0])


def _scan(B, N, C, S, G, dtype, seed):
    i = Inputs(seed, dtype)
    s = dict(u=i.normal(B, N, C), delta=i.normal(B, N, C, scale=0.5), A=-i.param(C, S).abs() - 0.5, Bm=i.normal(B, N, G, S),
             Cm=i.normal(B, N, G, S), D=i.param(C), delta_bias=i.param(C, mean=-3.0), z=i.normal(B, N, C))
    return s, i.normal(B, N, C), i.param(B, C, S)


NAMES = ("d_u", "d_delta", "d_A", "d_B", "d_C", "d_D", "d_delta_bias", "d_z", "d_h0")


@pytest.mark.parametrize("N,C,S,G,dtype", [(1, 64, 8, 1, "fp32"), (7, 70, 16, 1, "bf16"), (50, 66, 32, 2, "fp32"),
                                           (300, 64, 64, 1, "bf16"), (700, 40, 16, 1, "fp32")])
def test_scan_gradients_of_an_empty_sequence(N, C, S, G, dtype):
    """Its start state is in no product: whatever it holds, every gradient is that of a state of zeros, its own are zeros."""
    s, d_y, h0 = _scan(3, N, C, S, G, dtype, N + S)
    lengths = torch.tensor([N, 0, (N + 1) // 2], dtype=torch.int32, device="cuda")
    h0[1] = 0.0
    want = T.ttt_backward_selective_scan(**s, d_y=d_y, h0=h0, lengths=lengths)
    for value in (NAN, INF):
        h0[1] = value
        got = T.ttt_backward_selective_scan(**s, d_y=d_y, h0=h0, lengths=lengths)
        for name, g, r in zip(NAMES, got, want):
            assert torch.isfinite(r).all() and torch.equal(g, r), (name, value)
        assert not got[8][1].any()


@pytest.mark.parametrize("N,n,S,dtype", [(8, 3, 16, "bf16"), (40, 20, 8, "fp32"), (100, 64, 32, "bf16"), (90, 41, 64, "fp32")])
def test_scan_padding_behind_an_infinite_state(N, n, S, dtype):
    """A sequence whose states are infinite: its padding's rows of every gradient are zeros all the same."""
    s, d_y, h0 = _scan(2, N, 66, S, 1, dtype, N + S)
    h0[1, 5] = INF
    lengths = torch.tensor([N, n], dtype=torch.int32, device="cuda")
    got = dict(zip(NAMES, T.ttt_backward_selective_scan(**s, d_y=d_y, h0=h0, lengths=lengths)))
    for name in ("d_u", "d_delta", "d_B", "d_C", "d_z"):
        assert torch.isfinite(got[name][0]).all() and not got[name][1, n:].any(), name


@pytest.mark.parametrize("N,dtype", [(400, "fp32"), (3000, "bf16")])
def test_scan_states_of_zero_under_growing_decays(N, dtype):
    """step A = 8 a token: over a segment the decays' product is infinite, but states are zero until the last two tokens,
    where h = step B u and then exp(8) h + step B u. Off by the rounding of exp(8) (8 * 2 u + 2 u), of three products and
    of the sum over 8 states: 40 u of the sum of magnitudes, and the output's own rounding."""
    i = Inputs(N, dtype)
    C, S = 64, 8
    u, Bm, Cm = i.normal(1, N, C), i.normal(1, N, 1, S), i.normal(1, N, 1, S)
    u[:, :-2] = 0.0
    delta = torch.full((1, N, C), -4.0, dtype=DT[dtype], device="cuda")
    A = torch.full((C, S), -2.0, device="cuda")
    end = torch.empty(1, C, S, device="cuda")
    y = T.ttt_forward_selective_scan(u, delta, A, Bm, Cm, softplus=False, h_out=end)
    assert not y[:, :-2].any()
    drive = -4.0 * u[0, -2:].double()[..., None] * Bm[0, -2:].double()          # [2, C, S]
    last = 2.718281828459045 ** 8 * drive[0] + drive[1]
    most = 2.718281828459045 ** 8 * drive[0].abs() + drive[1].abs()
    unit = 2.0 ** -24
    assert ((end[0] - last).abs() <= 40 * unit * most).all()
    want, size = (last * Cm[0, -1].double()).sum(-1), (most * Cm[0, -1].double().abs()).sum(-1)
    assert ((y[0, -1] - want).abs() <= torch.finfo(DT[dtype]).eps / 2 * want.abs() + 40 * unit * size).all()
