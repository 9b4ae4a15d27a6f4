"""The float64 reference of tests/seq_reference.py against the oracle, on the CPU; and its bounds: an evaluation in fp32
keeps to them, one with an operand of 12 bits does not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import seq_reference as R  # noqa: E402
from oracle import seq_oracle as O  # noqa: E402


def _close(name, got, ref):
    scale = max(1e-300, np.abs(ref).max(initial=0.0))
    assert np.abs(got[0].numpy() - ref).max(initial=0.0) <= 1e-12 * scale, name
    assert (got[1].numpy() >= 0).all(), name


def _r(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


@pytest.mark.parametrize("shape", [(5, 7), (4, 3, 10), (2, 3, 1, 33)])
def test_layernorm_is_the_oracles(shape):
    w, b = _r(*shape[-2:] if len(shape) > 2 else shape[-1:], seed=1), _r(*shape[-2:] if len(shape) > 2 else shape[-1:], seed=2)
    x, d_y = _r(*shape), _r(*shape, seed=3)
    got = R.layernorm(x, w, b, d_y, 1e-5, 46, 10)
    n = lambda t: t.double().numpy()  # noqa: E731
    ref = dict(zip(("d_x", "d_weight", "d_bias"), O.layernorm_backward(n(x), n(w), n(d_y), 1e-5)), y=O.layernorm(n(x), n(w), n(b), 1e-5))
    for name, value in ref.items():
        _close(name, got[name], value)


@pytest.mark.parametrize("K,silu,state,lengths", [(2, True, True, [9, 0, 1]), (3, False, False, None), (4, True, True, [2, 9, 30]),
                                                  (4, False, True, [-1, 3, 9])])
def test_conv1d_is_the_oracles(K, silu, state, lengths):
    x, w, b, d_y = _r(3, 9, 5), _r(5, K, seed=1), _r(5, seed=2), _r(3, 9, 5, seed=3)
    s = _r(3, K - 1, 5, seed=4) if state else None
    n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    got = R.conv1d(x, w, b, d_y, silu, s, None if lengths is None else torch.tensor(lengths), 8)
    ref = dict(zip(("d_x", "d_weight", "d_bias", "d_state"), O.conv1d_backward(n(x), n(w), n(b), silu, n(d_y), n(s), lengths)))
    ref["y"] = O.conv1d(n(x), n(w), n(b), silu, n(s), lengths)[0]
    for name, value in ref.items():
        _close(name, got[name], value)


def _scan_inputs(B, N, C, S, G, gate, state, seed=0):
    k = iter(range(seed, seed + 20))
    r = lambda *s: _r(*s, seed=next(k))  # noqa: E731
    return dict(u=r(B, N, C), delta=r(B, N, C), A=-r(C, S).abs() - 0.05, Bm=r(B, N, G, S), Cm=r(B, N, G, S), D=r(C),
                delta_bias=r(C) - 2, z=r(B, N, C) if gate else None, h0=r(B, C, S) if state else None), r(B, N, C)


@pytest.mark.parametrize("gate,state,sp,lengths", [(True, True, True, [6, 0, 11]), (False, True, False, None), (True, False, True, [11, 40, -2])])
def test_scan_is_the_oracles(gate, state, sp, lengths):
    s, d_y = _scan_inputs(3, 11, 6, 8, 2, gate, state)
    if not sp:
        s["delta"], s["delta_bias"] = s["delta"].abs() * 0.1, None
    n = {k: None if v is None else v.double().numpy() for k, v in s.items()}
    n["dbias"] = n.pop("delta_bias")
    L = None if lengths is None else torch.tensor(lengths)
    got = R.scan(**s, softplus=sp, lengths=L)
    for name, value in zip(("y", "h_out"), O.scan(**n, sp=sp, lengths=lengths)):
        _close(name, got[name], value)
    got = R.scan(**s, d_y=d_y, softplus=sp, lengths=L)
    for name, value in O.scan_backward(**n, dy=d_y.double().numpy(), sp=sp, lengths=lengths).items():
        if name in got:
            _close(name, got[name], value)


def _fp32_scan(s, coarse=None):
    """y and h_out in fp32, token after token; `coarse` is an operand kept to 12 bits."""
    f = {k: None if v is None else v.clone() for k, v in s.items()}
    if coarse:
        f[coarse] = (f[coarse].view(torch.int32) & ~0xfff).view(torch.float32)
    h, ys = f["h0"].clone(), []
    for t in range(f["u"].shape[1]):
        dt = torch.nn.functional.softplus(f["delta"][:, t] + f["delta_bias"])[..., None]
        rep = f["u"].shape[2] // f["Bm"].shape[2]
        h = torch.exp(dt * f["A"]) * h + dt * f["u"][:, t, :, None] * f["Bm"][:, t].repeat_interleave(rep, 1)
        ys.append((f["Cm"][:, t].repeat_interleave(rep, 1) * h).sum(-1) + f["D"] * f["u"][:, t])
        ys[-1] = ys[-1] * (f["z"][:, t] * torch.sigmoid(f["z"][:, t]))
    return torch.stack(ys, 1), h


def test_scan_bounds_hold_for_fp32_and_not_for_12_bits():
    s, _ = _scan_inputs(2, 200, 16, 8, 1, True, True, seed=40)
    ref = R.scan(**s, tokens=1)
    for name, got in zip(("y", "h_out"), _fp32_scan(s)):
        assert R.held(name, got, ref[name]) <= 1.0
    for coarse in ("u", "delta", "Bm", "Cm", "z", "A"):
        with pytest.raises(AssertionError, match="times the bound"):
            R.held("y", _fp32_scan(s, coarse)[0], ref["y"])
