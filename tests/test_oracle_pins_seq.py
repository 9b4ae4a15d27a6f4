"""Pins of the fp64 oracle of the block operators (oracle/seq_oracle.py): closed forms, torch's own layer
norm and convolution, the scan's unrolled sum, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import seq_oracle as O

RNG = np.random.default_rng


def _differences(f, arrays, grads, names, h=1e-6, tol=1e-6):
    """Central differences of the scalar f(**arrays) at a few entries of each array."""
    rs = RNG(0)
    for name in names:
        a = arrays[name]
        for flat in rs.choice(a.size, size=min(a.size, 6), replace=False):
            at = np.unravel_index(flat, a.shape)
            keep = a[at]
            a[at] = keep + h
            up = f(**arrays)
            a[at] = keep - h
            down = f(**arrays)
            a[at] = keep
            want, got = (up - down) / (2 * h), grads[name][at]
            assert abs(want - got) <= tol * max(1.0, abs(want)), (name, at, want, got)


def test_layernorm_against_torch_and_differences():
    torch = pytest.importorskip("torch")
    rs = RNG(1)
    x, w, b, dy = rs.standard_normal((3, 5, 7)), rs.standard_normal(7), rs.standard_normal(7), rs.standard_normal((3, 5, 7))
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (7,), torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    assert np.allclose(O.layernorm(x, w, b, 1e-5), ref.numpy(), atol=1e-12)
    dx, dw, db = O.layernorm_backward(x, w, dy, 1e-5)
    _differences(lambda x, w, b: (O.layernorm(x, w, b, 1e-5) * dy).sum(), {"x": x, "w": w, "b": b},
                 {"x": dx, "w": dw, "b": db}, ("x", "w", "b"))


def test_layernorm_per_head_is_each_heads_own():
    rs = RNG(2)
    x, w, b, dy = rs.standard_normal((4, 3, 6)), rs.standard_normal((3, 6)), rs.standard_normal((3, 6)), rs.standard_normal((4, 3, 6))
    y, (dx, dw, db) = O.layernorm(x, w, b, 1e-3), O.layernorm_backward(x, w, dy, 1e-3)
    for h in range(3):
        assert np.allclose(y[:, h], O.layernorm(x[:, h], w[h], b[h], 1e-3))
        ex, ew, eb = O.layernorm_backward(x[:, h], w[h], dy[:, h], 1e-3)
        assert np.allclose(dx[:, h], ex) and np.allclose(dw[h], ew) and np.allclose(db[h], eb)


@pytest.mark.parametrize("K", [2, 3, 4])
def test_conv1d_against_torch(K):
    torch = pytest.importorskip("torch")
    rs = RNG(K)
    x, w, b = rs.standard_normal((2, 9, 5)), rs.standard_normal((5, K)), rs.standard_normal(5)
    pad = torch.nn.functional.pad(torch.from_numpy(x).transpose(1, 2), (K - 1, 0))
    ref = torch.nn.functional.conv1d(pad, torch.from_numpy(w)[:, None], torch.from_numpy(b), groups=5).transpose(1, 2)
    y, end = O.conv1d(x, w, b, False)
    assert np.allclose(y, ref.numpy(), atol=1e-12)
    assert np.allclose(end, x[:, -(K - 1):])
    assert np.allclose(O.conv1d(x, w, b, True)[0], torch.nn.functional.silu(ref).numpy(), atol=1e-12)


def test_conv1d_continues_from_its_state_and_stops_at_its_length():
    rs = RNG(5)
    x, w, b = rs.standard_normal((2, 9, 3)), rs.standard_normal((3, 4)), rs.standard_normal(3)
    whole = O.conv1d(x, w, b, True)[0]
    first, mid = O.conv1d(x[:, :2], w, b, True)
    second, _ = O.conv1d(x[:, 2:], w, b, True, state=mid)
    assert np.allclose(whole, np.concatenate([first, second], 1))
    y, end = O.conv1d(x, w, b, True, lengths=[2, 0])
    assert np.allclose(y[0, :2], whole[0, :2]) and not y[0, 2:].any() and not y[1].any()
    assert np.allclose(end[0], mid[0]) and not end[1].any()


@pytest.mark.parametrize("silu", [False, True])
def test_conv1d_gradients_against_differences(silu):
    rs = RNG(6)
    a = {"x": rs.standard_normal((2, 6, 3)), "w": rs.standard_normal((3, 4)), "b": rs.standard_normal(3),
         "state": rs.standard_normal((2, 3, 3))}
    dy, lengths = rs.standard_normal((2, 6, 3)), [6, 2]
    grads = dict(zip("x w b state".split(), O.conv1d_backward(a["x"], a["w"], a["b"], silu, dy, a["state"], lengths)))
    _differences(lambda x, w, b, state: (O.conv1d(x, w, b, silu, state, lengths)[0] * dy).sum(), a, grads, a)
    assert not grads["x"][1, 2:].any()


def test_scan_is_the_unrolled_sum():
    """h_t = sum_{j <= t} exp(A sum_{j < i <= t} step_i) step_j B_j u_j + exp(A sum_{i <= t} step_i) h0."""
    rs = RNG(7)
    B, N, C, S = 1, 7, 2, 3
    u, delta, Bm, Cm = rs.standard_normal((B, N, C)), rs.standard_normal((B, N, C)), rs.standard_normal((B, N, 1, S)), rs.standard_normal((B, N, 1, S))
    A, D, h0 = -np.exp(rs.standard_normal((C, S))), rs.standard_normal(C), rs.standard_normal((B, C, S))
    y, end = O.scan(u, delta, A, Bm, Cm, D, h0=h0)
    dt = np.log1p(np.exp(delta))
    for t in range(N):
        for c in range(C):
            h = np.exp(A[c] * dt[0, :t + 1, c].sum()) * h0[0, c]
            for j in range(t + 1):
                h = h + np.exp(A[c] * dt[0, j + 1:t + 1, c].sum()) * dt[0, j, c] * Bm[0, j, 0] * u[0, j, c]
            assert np.isclose(y[0, t, c], (Cm[0, t, 0] * h).sum() + D[c] * u[0, t, c])
        if t == N - 1:
            assert np.allclose(end[0, c], h)


def test_scan_continues_groups_and_lengths():
    rs = RNG(8)
    B, N, C, S, G = 2, 8, 4, 3, 2
    u, delta, z = (rs.standard_normal((B, N, C)) for _ in range(3))
    Bm, Cm = rs.standard_normal((B, N, G, S)), rs.standard_normal((B, N, G, S))
    A, D, db = -np.exp(rs.standard_normal((C, S))), rs.standard_normal(C), rs.standard_normal(C)
    whole, end = O.scan(u, delta, A, Bm, Cm, D, db, z)
    one, mid = O.scan(u[:, :3], delta[:, :3], A, Bm[:, :3], Cm[:, :3], D, db, z[:, :3])
    two, end2 = O.scan(u[:, 3:], delta[:, 3:], A, Bm[:, 3:], Cm[:, 3:], D, db, z[:, 3:], h0=mid)
    assert np.allclose(whole, np.concatenate([one, two], 1)) and np.allclose(end, end2)
    for g in range(G):  # a group's channels alone
        cs = slice(2 * g, 2 * g + 2)
        y, _ = O.scan(u[..., cs], delta[..., cs], A[cs], Bm[:, :, g:g + 1], Cm[:, :, g:g + 1], D[cs], db[cs], z[..., cs])
        assert np.allclose(y, whole[..., cs])
    y, e = O.scan(u, delta, A, Bm, Cm, D, db, z, lengths=[3, 0])
    assert np.allclose(y[0, :3], one[0]) and not y[0, 3:].any() and not y[1].any()
    assert np.allclose(e[0], mid[0]) and not e[1].any()


@pytest.mark.parametrize("sp,gate", [(True, True), (False, False)])
def test_scan_gradients_against_differences(sp, gate):
    rs = RNG(9)
    B, N, C, S, G = 2, 5, 4, 3, 2
    a = {"u": rs.standard_normal((B, N, C)), "delta": rs.standard_normal((B, N, C)),
         "A": -np.exp(rs.standard_normal((C, S))), "Bm": rs.standard_normal((B, N, G, S)),
         "Cm": rs.standard_normal((B, N, G, S)), "D": rs.standard_normal(C), "dbias": rs.standard_normal(C),
         "h0": rs.standard_normal((B, C, S))}
    if not sp:
        a["delta"], a["dbias"] = 0.1 * a["delta"], 0.1 * a["dbias"]
    if gate:
        a["z"] = rs.standard_normal((B, N, C))
    dy, lengths = rs.standard_normal((B, N, C)), [5, 3]
    got = O.scan_backward(dy=dy, sp=sp, lengths=lengths, **a)
    called = {"u": "d_u", "delta": "d_delta", "A": "d_A", "Bm": "d_B", "Cm": "d_C", "D": "d_D",
              "dbias": "d_delta_bias", "h0": "d_h0", "z": "d_z"}
    grads = {k: got[called[k]] for k in a}
    _differences(lambda **v: (O.scan(sp=sp, lengths=lengths, **v)[0] * dy).sum(), a, grads, a)
    assert not grads["u"][1, 3:].any() and not grads["Bm"][1, 3:].any()
