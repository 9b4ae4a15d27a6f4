"""GPU parity of layer norm, forward and backward, against the fp64 oracle (bounds: tests/seq_helpers.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_sequence_layers_amd as T
from oracle import seq_oracle as O
from seq_helpers import C_NORM, C_SUM, Inputs, check, f64, replays, sliced

EPS = 1e-5
CASES = [  # M, H, D, dtype, sliced
    (1, 1, 1, "fp32", False), (3, 1, 7, "bf16", False), (5, 1, 33, "fp32", True), (257, 1, 65, "bf16", False),
    (9, 12, 64, "bf16", False), (130, 12, 64, "bf16", True), (77, 3, 64, "fp32", False), (33, 5, 16, "bf16", False),
    (17, 2, 32, "fp32", True), (19, 40, 64, "bf16", False), (6, 7, 24, "bf16", True), (21, 3, 10, "fp32", False),
    (100, 1, 100, "bf16", False), (64, 1, 384, "bf16", False), (1, 1, 768, "bf16", False), (35, 1, 768, "fp32", True),
    (300, 1, 1001, "fp32", False), (41, 1, 1001, "bf16", True), (23, 1, 1280, "bf16", False), (10, 1, 2056, "bf16", False),
    (7, 1, 2050, "fp32", False), (12, 1, 4096, "fp32", False), (5, 2, 4100, "bf16", False), (9, 1, 8192, "bf16", True),
    (3, 1, 16384, "fp32", False), (3, 1, 16383, "bf16", False), (2, 1, 16384, "bf16", False), (5000, 1, 8, "fp32", False),
    (4100, 1, 128, "bf16", False), (3, 300, 8, "fp32", False),
]


def _inputs(M, H, D, dtype, cut, seed):
    i = Inputs(seed, dtype)
    shape = (M, H, D) if H > 1 else (M, D)
    x, d_y = i.normal(*shape, mean=0.5), i.normal(*shape)
    w, b = i.param(*shape[1:], scale=0.2, mean=1.0), i.param(*shape[1:], scale=0.3)
    # an extra of 8 elements keeps a slice's rows on 16 bytes, of 5 does not
    return (sliced(x, 1, 8 if D % 16 == 0 else 5) if cut else x), w, b, d_y


@pytest.mark.parametrize("M,H,D,dtype,cut", CASES, ids=lambda v: str(v))
def test_layernorm(M, H, D, dtype, cut):
    print(f"layernorm M={M} H={H} D={D} {dtype} sliced={cut}", flush=True)
    x, w, b, d_y = _inputs(M, H, D, dtype, cut, seed=M + 7 * D)
    y = T.ttt_forward_layernorm(x, w, b, EPS)
    dx, dw, db = T.ttt_backward_layernorm(x, w, d_y, EPS)
    torch.cuda.synchronize()
    check("y", y, O.layernorm(f64(x), f64(w), f64(b), EPS), C_NORM)
    if D > 1:  # of one channel xhat is 0, and dx what rounding leaves
        rx, rw, rb = O.layernorm_backward(f64(x), f64(w), f64(d_y), EPS)
        check("dx", dx, rx, C_NORM)
        check("dw", dw, rw, C_SUM)
        check("db", db, rb, C_SUM)
    else:
        assert not dx.any() and not dw.any()
        check("db", db, f64(d_y).sum(0), C_SUM)


def test_layernorm_without_bias_and_with_given_outputs():
    x, w, _, d_y = _inputs(37, 1, 192, "bf16", False, 3)
    y = torch.full_like(x, 7.0)
    assert T.ttt_forward_layernorm(x, w, eps=EPS, y=y) is y
    check("y", y, O.layernorm(f64(x), f64(w), None, EPS), C_NORM)
    outs = torch.full_like(x, 7.0), torch.full_like(w, 7.0), torch.full_like(w, 7.0)
    got = T.ttt_backward_layernorm(x, w, d_y, EPS, d_x=outs[0], d_weight=outs[1], d_bias=outs[2])
    assert all(a is b for a, b in zip(got, outs))
    for g, r, c in zip(got, O.layernorm_backward(f64(x), f64(w), f64(d_y), EPS), (C_NORM, C_SUM, C_SUM)):
        check("gradient", g, r, c)


def test_layernorm_far_mean_and_constant_rows():
    """fp32 rows 1000 deviations from zero: the mean is off by about 72 u of 1000, which the centred
    values carry at 72000 u of one deviation (2^-24 each), eight times that at the largest values. A
    constant row has variance 0: y is the bias up to x's own rounding times 1 / sqrt(eps)."""
    i = Inputs(11, "fp32")
    x, w, b = i.normal(20, 768, mean=1000.0), i.param(768, mean=1.0, scale=0.1), i.param(768)
    check("y", T.ttt_forward_layernorm(x, w, b, EPS), O.layernorm(f64(x), f64(w), f64(b), EPS), 8 * 72000)
    x = torch.full((4, 768), 2.0, device="cuda")
    assert torch.equal(T.ttt_forward_layernorm(x, w, b, EPS), b.expand(4, 768))


def test_layernorm_rows_with_infinities_stay_their_own():
    i = Inputs(12, "bf16")
    x, w, b = i.normal(6, 256), i.param(256), i.param(256)
    want = T.ttt_forward_layernorm(x, w, b, EPS)
    x[1, 3], x[4, 255] = float("inf"), float("nan")
    y = T.ttt_forward_layernorm(x, w, b, EPS)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], want[keep]) and torch.isnan(y[[1, 4]]).all()


def test_layernorm_aligned_and_unaligned_rows_agree():
    """The element-wise path against the 16-byte one on the same values."""
    i = Inputs(13, "bf16")
    x, w, b, d_y = i.normal(50, 512), i.param(512), i.param(512), i.normal(50, 512)
    off = sliced(x, 1, 3)
    a, c = T.ttt_forward_layernorm(x, w, b, EPS), T.ttt_forward_layernorm(off, w, b, EPS)
    ref = O.layernorm(f64(x), f64(w), f64(b), EPS)
    check("aligned", a, ref, C_NORM)
    check("unaligned", c, ref, C_NORM)
    for p, q, r, cc in zip(T.ttt_backward_layernorm(x, w, d_y, EPS), T.ttt_backward_layernorm(off, w, d_y, EPS),
                           O.layernorm_backward(f64(x), f64(w), f64(d_y), EPS), (C_NORM, C_SUM, C_SUM)):
        check("aligned", p, r, cc)
        check("unaligned", q, r, cc)


def test_layernorm_refuses_wrong_tensors():
    x, w = torch.zeros(4, 3, 8, device="cuda"), torch.zeros(3, 8, device="cuda")
    for bad in (dict(weight=torch.zeros(8, 3, device="cuda")), dict(weight=w.double()), dict(weight=w.t().contiguous().t()),
                dict(bias=torch.zeros(8, device="cuda")), dict(x=x.half()), dict(x=x.transpose(0, 1)),
                dict(x=torch.zeros(4, 3, 16, device="cuda")[..., ::2]), dict(y=torch.zeros(4, 24, device="cuda"))):
        args = dict(x=x, weight=w) | bad
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_layernorm(**args)
    with pytest.raises(T.TTTError):
        T.ttt_forward_layernorm(x, w, y=x)
    with pytest.raises(T.TTTError):
        T.ttt_forward_layernorm(x, w, eps=-1.0)


def test_layernorm_replayed_and_on_another_stream():
    x, w, b, d_y = _inputs(130, 12, 64, "bf16", True, 5)
    y, dx = torch.empty_like(d_y), torch.empty_like(d_y)
    dw, db = torch.empty_like(w), torch.empty_like(w)

    def call():
        T.ttt_forward_layernorm(x, w, b, EPS, y=y)
        T.ttt_backward_layernorm(x, w, d_y, EPS, d_x=dx, d_weight=dw, d_bias=db)

    replays(call, [y, dx, dw, db], lambda: T.ttt_forward_layernorm(d_y, w, b, EPS))
    want = [t.clone() for t in (y, dx, dw, db)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [T.ttt_forward_layernorm(x, w, b, EPS, stream=side), *T.ttt_backward_layernorm(x, w, d_y, EPS, stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
