"""Tensors that a block operator writes in place count as changed: autograd refuses a gradient that would take their old
values."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T


def _cases():
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, w, taps, A = r(2, 6, 16), r(16), r(16, 3), -r(16, 8).abs()
    Bm = r(2, 6, 1, 8)
    d_y, x1, b1 = r(2, 6, 16), x[:, 0].contiguous(), Bm[:, 0].contiguous()
    return [
        ("y", r(2, 6, 16), lambda t: T.ttt_forward_layernorm(x, w, y=t)),
        ("d_weight", r(16), lambda t: T.ttt_backward_layernorm(x, w, d_y, d_weight=t)),
        ("state_out", r(2, 2, 16), lambda t: T.ttt_forward_conv1d(x, taps, state_out=t)),
        ("state", r(2, 2, 16), lambda t: T.ttt_step_conv1d(x1, taps, state=t)),
        ("state_out of a step", r(2, 2, 16), lambda t: T.ttt_step_conv1d(x1, taps, state=r(2, 2, 16), state_out=t)),
        ("d_state", r(2, 2, 16), lambda t: T.ttt_backward_conv1d(x, taps, None, d_y, state=r(2, 2, 16), d_state=t)),
        ("h_out", r(2, 16, 8), lambda t: T.ttt_forward_selective_scan(x, x, A, Bm, Bm, h_out=t)),
        ("h", r(2, 16, 8), lambda t: T.ttt_step_selective_scan(x1, x1, A, b1, b1, h=t)),
        ("h_out of a step", r(2, 16, 8), lambda t: T.ttt_step_selective_scan(x1, x1, A, b1, b1, h=r(2, 16, 8), h_out=t)),
        ("d_h0", r(2, 16, 8), lambda t: T.ttt_backward_selective_scan(x, x, A, Bm, Bm, d_y, h0=r(2, 16, 8), d_h0=t)),
    ]


@pytest.mark.parametrize("k", range(10))
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


def test_inputs_do_not_count_as_changed_and_refused_calls_change_nothing():
    x, w = torch.randn(4, 16, device="cuda"), torch.randn(16, device="cuda")
    T.ttt_forward_layernorm(x, w)
    assert x._version == 0 and w._version == 0
    y = torch.empty_like(x)
    with pytest.raises(T.TTTError):
        T.ttt_forward_layernorm(x, w, eps=-1.0, y=y)
    assert y._version == 0


def test_states_of_inference_mode_are_taken():
    with torch.inference_mode():
        x, state = torch.randn(2, 16, device="cuda"), torch.zeros(2, 2, 16, device="cuda")
        T.ttt_step_conv1d(x, torch.ones(16, 3, device="cuda"), state=state)
        assert torch.equal(state[:, 1], x)
