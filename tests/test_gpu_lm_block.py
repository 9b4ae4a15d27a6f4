"""The residual block's operators together, as a language model uses them: the branch's dropout added to the residual stream and
normed at once, projections, the short convolution, the gated recurrence; forward, backward through torch's autograd, a prompt and then
single tokens, and the norm in 8 bits before a projection. Every stage is held to its own bound on the values that it was given.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
import seq_reference as Q  # noqa: E402
from lm_helpers import EPS, factors, rng_of  # noqa: E402
from seq_helpers import Inputs  # noqa: E402
from seq_reference import held  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

B, N, WIDTH, C, K, P = 2, 150, 96, 160, 4, 0.2
DEPTH = 46


class Norm(torch.autograd.Function):
    """(branch, residual, weight) -> (normed, sum), with dropout of the branch."""

    @staticmethod
    def forward(ctx, x, residual, w, rng):
        y, s = T.ttt_forward_rmsnorm(x, w, EPS, residual=residual, p=P, rng=rng)
        ctx.save_for_backward(s, w, rng)
        return y, s

    @staticmethod
    def backward(ctx, d_y, d_sum):
        s, w, rng = ctx.saved_tensors
        d_s, d_x, d_w = T.ttt_backward_rmsnorm(s, w, d_y.contiguous(), EPS, d_sum=d_sum.contiguous(), p=P, rng=rng)
        return d_x, d_s, d_w, None


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, lam, h0):
        kept = torch.empty(x.shape[0], (x.shape[1] + 63) // 64, x.shape[2], device=x.device)
        y = T.ttt_forward_gated_recurrence(x, r, i, lam, h0=h0, states=kept)
        ctx.save_for_backward(x, r, i, lam, h0, kept)
        return y

    @staticmethod
    def backward(ctx, d_y):
        x, r, i, lam, h0, kept = ctx.saved_tensors
        return T.ttt_backward_gated_recurrence(x, r, i, lam, d_y.contiguous(), h0=h0, states=kept)


def _weights(dtype):
    i = Inputs(5, dtype)
    w = {"norm": i.param(WIDTH, scale=0.1, mean=1.0), "w_in": i.normal(WIDTH, C, scale=WIDTH ** -0.5), "conv": i.param(C, K, scale=0.5),
         "w_gates": i.normal(C, 2 * C, scale=C ** -0.5), "lam": i.param(C, scale=1.0, mean=-4.0)}
    return i, w


def _reference_norm(x, res, w, f):
    s = x * f + res
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + EPS) * w, s


def _reference_recurrence(x, r, i, lam, h0):
    la = -8 * torch.nn.functional.softplus(lam) * torch.sigmoid(r)
    a, b = torch.exp(la), torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * x
    h, ys = h0, []
    for t in range(x.shape[1]):
        h = a[:, t] * h + b[:, t]
        ys.append(h)
    return torch.stack(ys, 1)


def test_gradients_through_a_block():
    """fp32, against autograd in float64 of the same block. The chain's outputs are off by at most some 2^-24 of their largest values
    for each of its stages' 2000 or so roundings in a row at gains below 10: 1e-4 of the largest."""
    i, w = _weights("fp32")
    rng, f = rng_of(3, 11), factors(3, 11, P, B * N, WIDTH).view(B, N, WIDTH)
    branch, residual, h0 = i.normal(B, N, WIDTH), i.normal(B, N, WIDTH), i.param(B, C)
    d_out, d_stream = i.normal(B, N, C), i.normal(B, N, WIDTH)
    leaves = [t.requires_grad_() for t in (branch, residual, w["norm"], w["w_in"], w["w_gates"], w["lam"], h0)]

    def block(norm, recurrence, branch, residual, wn, w_in, w_gates, lam, h0):
        y, s = norm(branch, residual, wn)
        u = y @ w_in
        gates = u @ w_gates
        return recurrence(u, gates[..., :C], gates[..., C:], lam, h0), s

    out, s = block(lambda x, r, v: Norm.apply(x, r, v, rng), Recurrence.apply, *leaves)
    grads = torch.autograd.grad((out, s), leaves, (d_out, d_stream))
    wide = [t.detach().double().requires_grad_() for t in leaves]
    ref, rs = block(lambda x, r, v: _reference_norm(x, r, v, f), _reference_recurrence, *wide)
    want = torch.autograd.grad((ref, rs), wide, (d_out.double(), d_stream.double()))
    for got, value in zip((out, s, *grads), (ref, rs, *want)):
        off = float((got.detach().double() - value.detach()).abs().max() / value.detach().abs().max())
        print(f"  {off:.2e}", flush=True)
        assert off < 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_prompt_then_single_tokens(dtype):
    """The whole sequence at once, and a prompt followed by tokens one at a time: each stage within its bound of float64 on the values
    that the library gave it, in both."""
    i, w = _weights(dtype)
    branch, residual, n0 = i.normal(B, N, WIDTH), i.normal(B, N, WIDTH), 131
    conv, h = i.normal(B, K - 1, C), i.param(B, C)
    conv0, h0 = conv.clone(), h.clone()

    def stages(x, res, last=False):
        y, s = T.ttt_forward_rmsnorm(x, w["norm"], EPS, residual=res)
        u = (y.float() @ w["w_in"].float()).to(i.io)
        v = T.ttt_step_conv1d(u, w["conv"], state=conv) if last else T.ttt_forward_conv1d(u, w["conv"], state=conv.clone(), state_out=conv)
        gates = (v.float() @ w["w_gates"].float()).to(i.io)
        r, g = gates[..., :C], gates[..., C:]
        if last:
            return y, s, u, v, gates, T.ttt_step_gated_recurrence(v, r, g, w["lam"], h=h)
        return y, s, u, v, gates, T.ttt_forward_gated_recurrence(v, r, g, w["lam"], h0=h.clone(), h_out=h)

    parts = [stages(branch[:, :n0].contiguous(), residual[:, :n0].contiguous())]
    parts += [tuple(t[:, None] for t in stages(branch[:, n].contiguous(), residual[:, n].contiguous(), True)) for n in range(n0, N)]
    y, s, u, v, gates, out = (torch.cat(t, 1) for t in zip(*parts))
    ref = R.rmsnorm(branch, w["norm"], EPS, DEPTH, residual)
    held("normed", y, ref["y"])
    held("sum", s, ref["sum"])
    held("convolved", v, Q.conv1d(u, w["conv"], None, state=conv0)["y"])
    ref = R.recurrence(v, gates[..., :C], gates[..., C:], w["lam"], h0=h0)
    held("out", out, ref["y"])
    held("state", h, ref["h_out"])
    assert torch.equal(conv, u[:, -(K - 1):])


def test_the_norm_in_8_bits_before_a_projection():
    """q (scales weights) against float64 of the exact norm: a product's terms are off by 2^-4 of them at most, of random sign, so that
    their sum of 96 is off by about 2^-4 / sqrt(3) of its standard deviation; five times that."""
    i, w = _weights("bf16")
    x, res = i.normal(B * N, WIDTH), i.normal(B * N, WIDTH)
    q, scales, s = T.ttt_forward_rmsnorm_e4m3(x, w["norm"], EPS, residual=res, group=32)
    got = (q.float().unflatten(-1, (-1, 32)) * scales[..., None]).flatten(-2) @ w["w_in"].float()
    y = R.rmsnorm(x, w["norm"], EPS, DEPTH, res)["y"][0]
    want = y @ w["w_in"].double()
    size = torch.sqrt(y.square() @ w["w_in"].double().square())
    assert float(((got.double() - want).abs() / size).max()) < 5 * 2.0 ** -4 / 3 ** 0.5
    assert torch.equal(s, (x.float() + res.float()).to(i.io))


def _cases():
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, w, rng = r(2, 70, 16), r(16), rng_of(1, 2)
    x1 = x[:, 0].contiguous()
    return [
        ("y", r(2, 70, 16), lambda t: T.ttt_forward_rmsnorm(x, w, y=t)),
        ("sum_out", r(2, 70, 16), lambda t: T.ttt_forward_rmsnorm(x, w, residual=x, sum_out=t)),
        ("residual in place", r(2, 70, 16), lambda t: T.ttt_forward_rmsnorm(x, w, residual=t, sum_out=t)),
        ("scales", r(2, 70, 1), lambda t: T.ttt_forward_rmsnorm_e4m3(x, w, scales=t)),
        ("d_x of a norm", r(2, 70, 16), lambda t: T.ttt_backward_rmsnorm(x, w, x, p=0.5, rng=rng, d_x=t)),
        ("d_sum in place", r(2, 70, 16), lambda t: T.ttt_backward_rmsnorm(x, w, x, d_sum=t, d_s=t)),
        ("dropped in place", r(2, 70, 16), lambda t: T.ttt_forward_dropout(t, 0.5, rng, y=t)),
        ("d_x", r(2, 70, 16), lambda t: T.ttt_backward_dropout(x, 0.5, rng, d_x=t)),
        ("h_out", r(2, 16), lambda t: T.ttt_forward_gated_recurrence(x, x, x, w, h_out=t)),
        ("states", r(2, 2, 16), lambda t: T.ttt_forward_gated_recurrence(x, x, x, w, states=t)),
        ("h", r(2, 16), lambda t: T.ttt_step_gated_recurrence(x1, x1, x1, w, h=t)),
        ("d_h0", r(2, 16), lambda t: T.ttt_backward_gated_recurrence(x, x, x, w, x, h0=r(2, 16), d_h0=t)),
    ]


@pytest.mark.parametrize("k", range(12))
def test_a_written_tensor_counts_as_changed(k):
    name, t, call = _cases()[k]
    print(name, flush=True)
    leaf = torch.ones_like(t, requires_grad=True)
    loss = (leaf * t).sum()  # (keeps t for leaf's gradient)
    before = t._version
    call(t)
    assert t._version > before, name
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_nothing_is_kept_and_inputs_are_left():
    import sys

    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, w, h, rng = r(2, 700, 64), r(64), r(2, 64), rng_of(1, 2)
    held_before = {"x": x.clone(), "w": w.clone(), "h": h.clone(), "rng": rng.clone()}

    def calls():
        y, s = T.ttt_forward_rmsnorm(x, w, residual=x, p=0.5, rng=rng)
        T.ttt_forward_rmsnorm_e4m3(x, w, residual=x)
        T.ttt_backward_rmsnorm(s, w, y, d_sum=x, p=0.5, rng=rng)
        T.ttt_backward_dropout(T.ttt_forward_dropout(x, 0.5, rng), 0.5, rng)
        T.ttt_backward_gated_recurrence(x, x, x, w, T.ttt_forward_gated_recurrence(x, x, x, w, h0=h), h0=h)
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_gated_recurrence(x, x, x, w[:4])
        with pytest.raises(T.TTTError):
            T.ttt_forward_dropout(x, 2.0, rng)

    calls()
    counts, memory = [sys.getrefcount(t) for t in (x, w, h, rng)], torch.cuda.memory_allocated()
    for _ in range(20):
        calls()
    assert [sys.getrefcount(t) for t in (x, w, h, rng)] == counts and torch.cuda.memory_allocated() == memory
    assert all(torch.equal(a, b) for a, b in zip((x, w, h, rng), held_before.values()))
    with torch.inference_mode():
        assert torch.equal(T.ttt_forward_rmsnorm(torch.nn.Parameter(x), torch.nn.Parameter(w)), T.ttt_forward_rmsnorm(x, w))


def test_calls_from_several_threads():
    """Each on a stream of its own, at once: the results of a call alone."""
    import threading

    cases = [(torch.randn(2, 1500 + 100 * k, 128, device="cuda"), torch.randn(128, device="cuda") - 4) for k in range(4)]
    want = [T.ttt_backward_gated_recurrence(x, x, x, lam, x) for x, lam in cases]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(cases))

    def work(k):
        try:
            stream, (x, lam) = torch.cuda.Stream(), cases[k]
            start.wait()
            for _ in range(30):
                got = T.ttt_backward_gated_recurrence(x, x, x, lam, x, stream=stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got[:4], want[k][:4])):
                bad.append(k)
        except Exception as e:  # noqa: BLE001
            bad.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
