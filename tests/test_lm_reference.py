"""The residual block's 64-bit references (CPU): the oracle's gradients against differences, the tests' reference against the
oracle, the generator against its published answers, e4m3 against a table of its numbers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lm_reference as R  # noqa: E402
from oracle import lm_oracle as O  # noqa: E402


def _rng(seed):
    return np.random.default_rng(seed)


def test_philox_gives_the_published_words():
    """The known answers published with the generator (10 rounds): counter and key of zeros, of ones, and of pi's digits."""
    ones = 0xFFFFFFFF
    assert O.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert O.philox4x32([ones] * 4, [ones] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert O.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_numbers_are_the_words_halves():
    seed, first = 0x0123456789ABCDEF, (1 << 64) - 2  # (the counter wraps)
    got = O.numbers(seed, first, 4)
    for j in range(4):
        at = (first + j) % (1 << 64)
        words = O.philox4x32([at & 0xFFFFFFFF, at >> 32, 0, 0], [seed & 0xFFFFFFFF, seed >> 32])
        assert got[j].tolist() == [h for w in words for h in (w & 0xFFFF, w >> 16)]


@pytest.mark.parametrize("p", [0.1, 0.25, 0.5, 0.9])
def test_masks_drop_about_p(p):
    """2^20 elements: the share kept is 1 - p' to five deviations."""
    f = O.factors(7, 3, p, 1024, 1024)
    q = 1 - np.rint(p * 65536) / 65536
    assert abs((f > 0).mean() - q) < 5 * np.sqrt(q * (1 - q) / f.size)
    assert abs(f.mean() - 1) < 5 * np.sqrt((1 - q) / q / f.size)


def test_e4m3_numbers():
    table = sorted({s * (1 + f / 8) * 2.0 ** e for s in (-1, 1) for e in range(-6, 9) for f in range(8)} |
                   {s * f * 2.0 ** -9 for s in (-1, 1) for f in range(8)})
    table = np.array([v for v in table if abs(v) <= 448])
    assert len(table) == 2 * (15 * 8 - 1) + 15  # (480 is not a number; zero once)
    assert np.array_equal(O.e4m3(table), table)
    v = np.concatenate([_rng(0).uniform(-448, 448, 20000), _rng(1).normal(0, 0.02, 20000)])
    assert np.array_equal(np.abs(O.e4m3(v) - v), np.abs(v[:, None] - table).min(1))
    assert O.e4m3(np.array([17.0, 19.0, 2.0 ** -10])).tolist() == [16.0, 20.0, 0.0]
    t = torch.tensor(v, dtype=torch.float32)
    assert np.array_equal(t.to(torch.float8_e4m3fn).double().numpy(), O.e4m3(t.double().numpy()))


def _differences(f, x, d_out, h=1e-6):
    """Central differences of sum(f(x) d_out) by every entry of x."""
    g = np.zeros_like(x)
    for at in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        g[at] = ((f(up) - f(down)) * d_out).sum() / (2 * h)
    return g


def test_rmsnorm_gradients_by_differences():
    rng = _rng(2)
    s, w, d_y, d_sum = rng.normal(size=(3, 2, 5)), rng.normal(size=(2, 5)), rng.normal(size=(3, 2, 5)), rng.normal(size=(3, 2, 5))
    d_s, d_w = O.rmsnorm_backward(s, w, d_y, 1e-3, d_sum)
    assert np.allclose(d_s - d_sum, _differences(lambda v: O.rmsnorm(v, w, 1e-3), s, d_y), atol=1e-8)
    assert np.allclose(d_w, _differences(lambda v: O.rmsnorm(s, v, 1e-3), w, d_y), atol=1e-8)


@pytest.mark.parametrize("lengths", [None, [7, 4]])
def test_recurrence_gradients_by_differences(lengths):
    rng = _rng(3)
    B, N, C = 2, 7, 3
    x, r, i, d_y = (rng.normal(size=(B, N, C)) for _ in range(4))
    lam, h0 = rng.normal(size=C) - 2, rng.normal(size=(B, C))
    got = O.recurrence_backward(x, r, i, lam, d_y, 8.0, h0, lengths)
    args = {"x": x, "r": r, "i": i, "lam": lam, "h0": h0}
    for k in args:
        f = lambda v, k=k: O.recurrence(**(args | {k: v}), scale=8.0, lengths=lengths)[0]  # noqa: E731
        assert np.allclose(got["d_" + k], _differences(f, args[k], d_y), atol=1e-7), k


def _t(a):
    return None if a is None else torch.from_numpy(np.asarray(a))


def _same(got, want, name):
    assert np.allclose(got[0].numpy(), want, rtol=1e-10, atol=1e-12), name
    assert float((got[1] - 1e-4 * (got[0].abs() + got[0].abs().max())).max()) <= 0 and float(got[1].min()) >= 0, name


def test_the_tests_reference_is_the_oracle():
    """Its values; and its bounds are small beside them (1e-4 of the largest) and not negative."""
    rng = _rng(4)
    x, res, w, d_y, d_sum = (rng.normal(size=(6, 40)) for _ in range(5))
    w, f = w[0], O.factors(11, 5, 0.3, 6, 40)
    ref = R.rmsnorm(_t(x), _t(w), 1e-5, 46, _t(res), _t(f))
    _same(ref["sum"], x * f + res, "sum")
    _same(ref["y"], O.rmsnorm(x * f + res, w, 1e-5), "y")
    back = R.rmsnorm_backward(_t(x), _t(w), _t(d_y), 1e-5, 46, 10, _t(d_sum), _t(f))
    d_s, d_w = O.rmsnorm_backward(x, w, d_y, 1e-5, d_sum)
    _same(back["d_s"], d_s, "d_s")
    _same(back["d_x"], d_s * f, "d_x")
    _same(back["d_weight"], d_w, "d_weight")
    B, N, C = 2, 30, 5
    x, r, i, d_y = (rng.normal(size=(B, N, C)) for _ in range(4))
    lam, h0 = rng.normal(size=C) - 3, rng.normal(size=(B, C))
    for lengths in (None, [30, 11]):
        t = None if lengths is None else torch.tensor(lengths)
        ref = R.recurrence(_t(x), _t(r), _t(i), _t(lam), h0=_t(h0), lengths=t)
        y, end, before = O.recurrence(x, r, i, lam, 8.0, h0, lengths)
        _same(ref["y"], y, "y")
        _same(ref["h_out"], end, "h_out")
        _same(ref["before"], before, "before")
        back = R.recurrence(_t(x), _t(r), _t(i), _t(lam), _t(d_y), h0=_t(h0), lengths=t)
        for k, v in O.recurrence_backward(x, r, i, lam, d_y, 8.0, h0, lengths).items():
            _same(back[k], v, k)


def test_a_planted_mistake_is_outside_the_bound():
    """A decay kept to bf16, and a state one token late, are off by more than the bounds."""
    rng = _rng(5)
    B, N, C = 1, 200, 8
    x, r, i = (rng.normal(size=(B, N, C)) for _ in range(3))
    lam = np.full(C, -4.0)
    y, bound = R.recurrence(_t(x), _t(r), _t(i), _t(lam))["y"]
    la = -8 * O.softplus(lam) * O.sigmoid(r)
    a = _t(np.exp(la)).to(torch.bfloat16).double()
    b = _t(np.sqrt(-np.expm1(2 * la)) * O.sigmoid(i) * x)
    h, worst = torch.zeros(B, C, dtype=torch.float64), 0.0
    for n in range(N):
        h = a[:, n] * h + b[:, n]
        worst = max(worst, float(((h - y[:, n]).abs() / (bound[:, n] + 2.0 ** -9 * y[:, n].abs())).max()))
    assert worst > 2
    assert float(((y[:, 1:] - y[:, :-1]).abs() / (bound[:, 1:] + 2.0 ** -9 * y[:, 1:].abs())).median()) > 10
