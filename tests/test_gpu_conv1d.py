"""GPU parity of the short causal convolution, forward, backward and single tokens, against the fp64
oracle (bounds: tests/seq_helpers.py)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T
from oracle import seq_oracle as O
from seq_helpers import C_CONV, C_SUM, Inputs, check, f64, replays, sliced

CASES = [  # B, N, C, K, dtype, silu, bias, state, lengths, sliced
    (1, 1, 1, 2, "fp32", False, False, False, None, False),
    (2, 1, 8, 4, "bf16", True, True, True, None, False),
    (2, 2, 16, 4, "bf16", True, True, False, None, True),
    (1, 3, 5, 4, "fp32", True, True, True, [2], False),
    (3, 15, 24, 3, "bf16", True, True, True, [0, 1, 15], False),
    (1, 16, 768, 4, "bf16", True, True, False, None, True),
    (2, 17, 193, 4, "bf16", True, True, True, None, True),
    (2, 33, 193, 2, "fp32", False, True, True, [33, 5], False),
    (3, 127, 40, 4, "fp32", True, False, True, [127, 64, 16], True),
    (1, 128, 64, 3, "bf16", False, True, False, None, False),
    (2, 129, 264, 4, "bf16", True, True, True, [129, 128], False),
    (4, 300, 100, 4, "fp32", True, True, True, [300, -5, 1000, 17], False),
    (2, 1000, 768, 4, "bf16", True, True, False, None, False),
    (1, 2049, 36, 4, "fp32", True, True, True, None, True),
]


def _inputs(B, N, C, K, dtype, bias, state, lengths, cut, seed):
    i = Inputs(seed, dtype)
    x, d_y = i.normal(B, N, C), i.normal(B, N, C)
    w, b = i.param(C, K, scale=K ** -0.5), i.param(C, scale=0.2) if bias else None
    st = i.normal(B, K - 1, C) if state else None
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths else None
    if lengths:  # padding holds anything
        for j, n in enumerate(lengths):
            x[j, max(n, 0):], d_y[j, max(n, 0):] = float("nan"), float("inf")
    return (sliced(x, 2, 8 if C % 8 == 0 else 5) if cut else x), d_y, w, b, st, ln


@pytest.mark.parametrize("B,N,C,K,dtype,silu,bias,state,lengths,cut", CASES, ids=lambda v: str(v))
def test_conv1d(B, N, C, K, dtype, silu, bias, state, lengths, cut):
    print(f"conv1d B={B} N={N} C={C} K={K} {dtype} silu={silu} lengths={lengths}", flush=True)
    x, d_y, w, b, st, ln = _inputs(B, N, C, K, dtype, bias, state, lengths, cut, seed=N + 3 * C)
    end = torch.full((B, K - 1, C), 7.0, device="cuda", dtype=x.dtype)
    y = T.ttt_forward_conv1d(x, w, b, silu=silu, state=st, lengths=ln, state_out=end)
    got = T.ttt_backward_conv1d(x, w, b, d_y, silu=silu, state=st, lengths=ln)
    torch.cuda.synchronize()
    ry, rend = O.conv1d(f64(x), f64(w), f64(b), silu, f64(st), lengths)
    check("y", y, ry, C_CONV)
    check("state_out", end, rend, 0)
    refs = O.conv1d_backward(f64(x), f64(w), f64(b), silu, f64(d_y), f64(st), lengths)
    for name, g, r, c in zip(("dx", "dw", "db", "dstate"), got, refs, (C_CONV, C_SUM, C_SUM, C_CONV)):
        if g is not None:
            check(name, g, r, c)
    assert (got[2] is None) == (b is None) and (got[3] is None) == (st is None)


@pytest.mark.parametrize("dtype,C,K", [("bf16", 64, 4), ("fp32", 19, 3), ("bf16", 7, 2)])
def test_conv1d_tokens_continue_a_prompt(dtype, C, K):
    """A prompt with its state kept, then single tokens in place, against the whole sequence at once: the
    same inputs meet the same arithmetic, so the bits agree."""
    i = Inputs(C, dtype)
    B, N, M = 3, 10, 6
    x, w, b = i.normal(B, N + M, C), i.param(C, K), i.param(C)
    whole = T.ttt_forward_conv1d(x, w, b, silu=True)
    state = torch.empty(B, K - 1, C, device="cuda", dtype=x.dtype)
    y = T.ttt_forward_conv1d(x[:, :N], w, b, silu=True, state_out=state) if B == 1 else T.ttt_forward_conv1d(
        x[:, :N].contiguous(), w, b, silu=True, state_out=state)
    assert torch.equal(y, whole[:, :N])
    for t in range(N, N + M):
        if t % 2:
            y = T.ttt_step_conv1d(x[:, t], w, b, silu=True, state=state)
        else:
            out = torch.empty_like(state)
            y = T.ttt_step_conv1d(x[:, t], w, b, silu=True, state=state, state_out=out)
            state = out
        assert torch.equal(y, whole[:, t])
    assert torch.equal(state, x[:, -(K - 1):])
    second = T.ttt_forward_conv1d(x[:, N:].contiguous(), w, b, silu=True, state=x[:, N - K + 1:N].contiguous())
    assert torch.equal(second, whole[:, N:])


def test_conv1d_large_values_saturate():
    """SiLU far from zero: sigmoid is 0 or 1, nothing overflows into NaN."""
    x = torch.tensor([-1e30, -200.0, 200.0, 1e30], device="cuda").view(1, 4, 1).repeat(1, 1, 8)
    w = torch.zeros(8, 4, device="cuda")
    w[:, 3] = 1.0
    y = T.ttt_forward_conv1d(x, w, silu=True)
    assert torch.equal(y[0, :, 0], torch.tensor([0.0, 0.0, 200.0, 1e30], device="cuda"))
    dx, _, _, _ = T.ttt_backward_conv1d(x, w, None, torch.ones_like(x), silu=True)
    assert torch.isfinite(dx).all()


def test_conv1d_refuses_wrong_tensors():
    x, w = torch.zeros(2, 5, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    for bad in (dict(x=x[:, :, :4]), dict(x=x.transpose(1, 2)), dict(x=x[:, ::2, ::2]), dict(weight=w.t()),
                dict(bias=torch.zeros(4, device="cuda")), dict(state=torch.zeros(2, 4, 8, device="cuda")),
                dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(state=torch.zeros(2, 3, 8, device="cuda", dtype=torch.bfloat16)), dict(x=x[:, :3])):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_conv1d(**(dict(x=x, weight=w) | bad))
    with pytest.raises(T.TTTError):
        T.ttt_forward_conv1d(x, torch.zeros(8, 5, device="cuda"))
    with pytest.raises(T.TTTError):
        T.ttt_forward_conv1d(x, w, y=x)
    state = torch.zeros(2, 3, 8, device="cuda")
    with pytest.raises(T.TTTError):  # the forward's states do not overlap; a step's may be the same
        T.ttt_forward_conv1d(x, w, state=state, state_out=state)
    with pytest.raises(ValueError):
        T.ttt_backward_conv1d(x, w, None, x, d_bias=torch.zeros(8, device="cuda"))


def test_conv1d_replayed_and_on_another_stream():
    x, d_y, w, b, st, ln = _inputs(2, 129, 264, 4, "bf16", True, True, [129, 100], True, 4)
    y, dx, ds = torch.empty_like(d_y), torch.empty_like(d_y), torch.empty_like(st)
    dw, db, end = torch.empty_like(w), torch.empty_like(b), torch.empty_like(st)

    def call():
        T.ttt_forward_conv1d(x, w, b, silu=True, state=st, lengths=ln, state_out=end, y=y)
        T.ttt_backward_conv1d(x, w, b, d_y, silu=True, state=st, lengths=ln, d_x=dx, d_weight=dw, d_bias=db, d_state=ds)

    replays(call, [y, end, dx, dw, db, ds], lambda: T.ttt_forward_conv1d(y, w, b))
    want = [t.clone() for t in (y, dx, dw, db, ds)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [T.ttt_forward_conv1d(x, w, b, silu=True, state=st, lengths=ln, stream=side),
           *T.ttt_backward_conv1d(x, w, b, d_y, silu=True, state=st, lengths=ln, stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B,N,C,dtype", [(2, 2049, 1028, "bf16"), (3, 4097, 1000, "fp32"), (2, 8193, 1032, "bf16")])
def test_conv1d_long_runs(B, N, C, dtype):
    """The sizes from which a thread walks 8, 16 and 32 tokens."""
    print(f"conv1d B={B} N={N} C={C} {dtype}", flush=True)
    x, d_y, w, b, st, ln = _inputs(B, N, C, 4, dtype, True, True, [N, N - 37, 5][:B], False, seed=N)
    lengths = [N, N - 37, 5][:B]
    end = torch.empty_like(st)
    y = T.ttt_forward_conv1d(x, w, b, silu=True, state=st, lengths=ln, state_out=end)
    got = T.ttt_backward_conv1d(x, w, b, d_y, silu=True, state=st, lengths=ln)
    torch.cuda.synchronize()
    ry, rend = O.conv1d(f64(x), f64(w), f64(b), True, f64(st), lengths)
    check("y", y, ry, C_CONV)
    check("state_out", end, rend, 0)
    refs = O.conv1d_backward(f64(x), f64(w), f64(b), True, f64(d_y), f64(st), lengths)
    for name, g, r, c in zip(("dx", "dw", "db", "dstate"), got, refs, (C_CONV, C_SUM, C_SUM, C_CONV)):
        check(name, g, r, c)
