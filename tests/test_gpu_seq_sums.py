"""The block operators' sums where fp32 loses the most: rows far from zero, sums over very many tokens."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T
from oracle import seq_oracle as O
from seq_helpers import Inputs, U, f64

EPS = 1e-5


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H,D,dtype", [(1, 64, "fp32"), (12, 64, "fp32"), (1, 300, "fp32"), (1, 768, "fp32"), (1, 1001, "fp32"),
                                       (1, 1001, "bf16"), (1, 4096, "fp32"), (1, 4100, "fp32"), (1, 16384, "fp32")])
def test_layernorm_of_constant_rows_is_the_bias(H, D, dtype):
    """x - mean is 0 whatever the row's value: y is the bias, d_x is rstd (g - mean(g)), d_weight 0."""
    i = Inputs(D, dtype)
    shape = (H, D) if H > 1 else (D,)
    values = torch.tensor([0.1, -7.3, 1000.1, 1000000.5, -3.3e7, 1e-20], device="cuda").to(i.io)
    x = values.view(-1, *[1] * len(shape)).expand(-1, *shape).contiguous()
    w, b, d_y = i.param(*shape, mean=1.0), i.param(*shape), i.normal(*x.shape)
    assert torch.equal(T.ttt_forward_layernorm(x, w, b, EPS), b.expand_as(x).to(i.io))
    dx, dw, _ = T.ttt_backward_layernorm(x, w, d_y, EPS)
    assert not dw.any() and torch.isfinite(dx).all()


@pytest.mark.parametrize("D,dtype,sliced", [(64, "fp32", 0), (768, "fp32", 0), (768, "fp32", 1), (2050, "fp32", 0), (4096, "fp32", 0)])
def test_layernorm_of_rows_far_from_zero(D, dtype, sliced):
    """Rows 1e5 deviations from zero. x is exact, and only differences of its elements enter: with |x - mean| <= 5
    deviations (asserted), a difference x - x' is off by u times 10 deviations, and the mean of D of them by as much and by 72 u
    (at most 64 terms in a lane and 8 levels) of their mean magnitude, at most 6: below 450 u of a deviation, in xhat and,
    twice, relatively in rstd: |y - ref| <= u |ref| + 450 u (1 + 2 * 5) |w| + 4 u |b|, the result's own rounding first."""
    i = Inputs(D, dtype)
    w, b = i.param(D, mean=1.0, scale=0.2), i.param(D)
    x = i.normal(20, D).clamp_(-4, 4) + 1e5
    if sliced:
        x = torch.cat([x, x], 1)[:, 1:1 + D]
    ref = O.layernorm(f64(x), f64(w), f64(b), EPS)
    dev = f64(x) - f64(x).mean(-1, keepdims=True)
    assert np.abs(dev).max() <= 5 * dev.std(-1).min()
    got = f64(T.ttt_forward_layernorm(x, w, b, EPS))
    bound = U * np.abs(ref) + 450 * 11 * U * np.abs(f64(w)) + 4 * U * np.abs(f64(b))
    worst = (np.abs(got - ref) / bound).max()
    print(f"  {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0


def test_scan_gradients_of_very_long_sequences():
    """4096 sequences of one channel, 32768 tokens each: as many blocks of channels as segments are wanted. All inputs
    constant, so that every sum is known, and one by one in fp32 it would drift (32768 times 0.003: 98.27 for 98.30,
    5900 u). Partial sums of at most 2048 tokens, each addition off by at most u of what is held, 65536 of them added
    1024 in a row and 6 levels: d_D within 3200 u. d_C is v h: h = exp(A sum step), |A| sum step <= 6.6, the sum of a segment's
    2048 steps within 2048 u and 15 segments' decays multiplied, and 2 u and an exponential each token of the last: (2048 +
    2) 6.6 + 2 * 2048 + 2 * 15 u < 18000 u."""
    B, N, S = 4096, 32768, 8
    full = lambda value, *shape: torch.full(shape, value, device="cuda")  # noqa: E731
    u, delta, v, a = 0.06, 0.003, 0.05, -0.067
    d_y = full(v, B, N, 1)
    got = T.ttt_backward_selective_scan(full(u, B, N, 1), full(delta, B, N, 1), full(a, 1, S), torch.zeros(B, N, 1, S, device="cuda"),
                                        torch.zeros(B, N, 1, S, device="cuda"), d_y, torch.ones(1, device="cuda"),
                                        softplus=False, h0=torch.ones(B, 1, S, device="cuda"))
    r = np.float32
    v, u, delta, a = (float(r(q)) for q in (v, u, delta, a))
    d_D, want = float(got[5]), B * N * v * u
    print(f"  d_D {d_D:.6g}, {want:.6g}: off by {abs(d_D / want - 1) / U:.0f} u", flush=True)
    d_C = got[4][::512, :, 0, :].double()
    h = torch.exp(a * delta * torch.arange(1, N + 1, device="cuda", dtype=torch.float64))[None, :, None]
    off = float((d_C / (v * h) - 1).abs().max())
    print(f"  d_C off by {off / U:.0f} u", flush=True)
    assert abs(d_D / want - 1) <= 3200 * U
    assert off <= 18000 * U


def test_layernorm_gradients_of_many_heads_and_rows():
    """4096 heads, as many workgroups as the backward pass wants, and 32768 tokens of d_y = 0.77: one after the other fp32 is
    3300 u off. A group of lanes walks at most 2048 turns, 16 groups and the partial rows follow: within 2200 u."""
    H, M = 4096, 32768
    x, d_y = torch.zeros(M, H, 1, device="cuda"), torch.full((M, H, 1), 0.77, device="cuda")
    d_bias = T.ttt_backward_layernorm(x, torch.ones(H, 1, device="cuda"), d_y)[2]
    off = float((d_bias.double() / (M * float(np.float32(0.77))) - 1).abs().max())
    print(f"  off by {off / U:.0f} u", flush=True)
    assert off <= 2200 * U


def test_scan_gradients_of_very_many_channels():
    """d_B and d_C of 2^20 channels whose products are all 0.77: blocks of 64 without rounding, then 16384 blocks, 64 at a
    time: 64 and 256 additions and a few more, 350 u. (One after the other they are 3300 u off.)"""
    C, S = 1 << 20, 8
    one = lambda *shape: torch.ones(*shape, device="cuda")  # noqa: E731
    got = T.ttt_backward_selective_scan(one(1, 1, C), one(1, 1, C), torch.zeros(C, S, device="cuda"), one(1, 1, 1, S), one(1, 1, 1, S),
                                        0.77 * one(1, 1, C), softplus=False)
    for name, t in (("d_B", got[3]), ("d_C", got[4])):
        off = float((t.double() / (C * float(np.float32(0.77))) - 1).abs().max())
        print(f"  {name} off by {off / U:.0f} u", flush=True)
        assert off <= 350 * U, name


def test_conv1d_gradients_of_very_many_tokens():
    """d_bias of 2^28 tokens of 0.77: runs of 32 tokens, 8 of a workgroup, and 2^20 partial rows, 64 threads to a column with
    2048 sums of 8 each and 6 levels: within 2110 u. (16384 rows one after the other are 3300 u off.)"""
    B, N, C = 64, 1 << 22, 4
    x, d_y = torch.zeros(B, N, C, device="cuda"), torch.full((B, N, C), 0.77, device="cuda")
    d_bias = T.ttt_backward_conv1d(x, torch.ones(C, 4, device="cuda"), torch.zeros(C, device="cuda"), d_y)[2]
    off = float((d_bias.double() / (B * N * float(np.float32(0.77))) - 1).abs().max())
    print(f"  off by {off / U:.0f} u", flush=True)
    assert off <= 2110 * U
