"""Dropout against the generator in integers and the sum in float64: masks to the bit, values within their roundings."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
from lm_helpers import factors, rng_of  # noqa: E402
from seq_helpers import Inputs, replays, sliced  # noqa: E402
from seq_reference import held  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

CASES = [  # shape, dtype, p, extra elements of a slice (None: contiguous)
    ((1, 1), "fp32", 0.5, None), ((1, 8), "bf16", 0.1, None), ((3, 7), "bf16", 0.25, None), ((5, 17), "fp32", 0.9, None),
    ((257, 64), "bf16", 0.1, None), ((12, 384), "fp32", 0.1, None), ((300, 1001), "fp32", 0.25, None), ((41, 513), "bf16", 0.5, None),
    ((33, 512), "bf16", 0.1, 5), ((33, 512), "bf16", 0.1, 8), ((20, 24), "fp32", 0.3, 4), ((7, 1100), "bf16", 0.3, 3),
    ((2, 3, 5, 40), "bf16", 0.3, None), ((1, 100000), "bf16", 0.1, None), ((3000, 384), "bf16", 0.1, None), ((9, 4097), "fp32", 0.7, None),
    ((64,), "bf16", 0.5, None),
]
SEED, OFFSET = (1 << 63) + 12345, (1 << 64) - 3  # (offsets wrap)


def _flat(shape):
    n = 1
    for v in shape[:-1]:
        n *= v
    return n, shape[-1]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_dropout(case, add):
    shape, dtype, p, extra = case
    print(f"dropout {shape} {dtype} p={p} extra={extra} residual={add}", flush=True)
    i = Inputs(shape[-1], dtype)
    x, res, d_y = i.normal(*shape), i.normal(*shape) if add else None, i.normal(*shape)
    x = x if extra is None else sliced(x, len(shape) - 1, extra)
    rng, f = rng_of(SEED, OFFSET), factors(SEED, OFFSET, p, *_flat(shape)).view(shape)
    y = T.ttt_forward_dropout(x, p, rng, residual=res)
    held("y", y, R.dropout(x, f, res))
    if not add:
        assert torch.equal(y != 0, (f > 0) & (x != 0))
    d_x = T.ttt_backward_dropout(d_y, p, rng)
    held("d_x", d_x, R.dropout(d_y, f))
    assert torch.equal(d_x != 0, (f > 0) & (d_y != 0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_narrow_width_at_every_alignment(dtype):
    for C in [*range(1, 26), 511, 513]:
        i = Inputs(C, dtype)
        e = C % 8
        x, res, f = sliced(i.normal(9, C), 1, e), i.normal(9, C), factors(SEED, OFFSET, 0.5, 9, C)
        around = torch.full((9 * C + 32,), 7.0, dtype=i.io, device="cuda")
        y = around[8 + e:8 + e + 9 * C].view(9, C)
        T.ttt_forward_dropout(x, 0.5, rng_of(SEED, OFFSET), residual=res, y=y)
        held(f"y of {C}", y, R.dropout(x, f, res))
        assert bool((around[:8 + e] == 7).all()) and bool((around[8 + e + 9 * C:] == 7).all())


def test_the_mask_is_the_norms():
    """A call of its own, of rows or one of many, drops what the fused one does."""
    i = Inputs(1, "fp32")
    for C in (768, 1001):
        x, res, w = i.normal(50, C), i.normal(50, C), i.param(C)
        rng = rng_of(3, 4)
        s = T.ttt_forward_rmsnorm(x, w, residual=res, p=0.4, rng=rng)[1]
        y = T.ttt_forward_dropout(x, 0.4, rng, residual=res)
        assert torch.equal(s != res, y != res) and torch.equal(s, y)


def test_offsets_follow_on():
    """A mask of rows 10 .. 30 is that of all rows, from the counters of the first ten on."""
    x = torch.ones(30, 100, device="cuda")
    rng = rng_of(8, 1000)
    whole = T.ttt_forward_dropout(x, 0.5, rng)
    assert T.dropout_counters(x[:10]) == 130
    rng[1] += T.dropout_counters(x[:10])
    assert torch.equal(T.ttt_forward_dropout(x[10:].contiguous(), 0.5, rng), whole[10:])


def test_no_probability_and_dropped_values():
    i = Inputs(2, "bf16")
    x, res = i.normal(9, 72), i.normal(9, 72)
    assert torch.equal(T.ttt_forward_dropout(x, 0.0, None), x)
    assert torch.equal(T.ttt_forward_dropout(x, 0.0, None, residual=res), (x.float() + res.float()).bfloat16())
    rng, f = rng_of(0, 0), factors(0, 0, 0.5, 9, 72)
    want = T.ttt_forward_dropout(x, 0.5, rng)
    bad = x.clone()
    bad[f == 0] = float("inf")
    assert torch.equal(T.ttt_forward_dropout(bad, 0.5, rng), want)
    odd = bad[:, :71].contiguous()
    assert torch.isfinite(T.ttt_forward_dropout(odd, 0.5, rng)[factors(0, 0, 0.5, 9, 71) == 0]).all()


@pytest.mark.parametrize("C", [768, 771])
def test_in_place(C):
    i = Inputs(C, "bf16")
    x, res, rng = i.normal(64, C), i.normal(64, C), rng_of(5, 6)
    want, both = T.ttt_forward_dropout(x, 0.3, rng), T.ttt_forward_dropout(x, 0.3, rng, residual=res)
    a, b, c = x.clone(), res.clone(), x.clone()
    assert T.ttt_forward_dropout(a, 0.3, rng, y=a) is a and torch.equal(a, want) and a._version > 0
    assert torch.equal(T.ttt_forward_dropout(x, 0.3, rng, residual=b, y=b), both)
    assert torch.equal(T.ttt_backward_dropout(c, 0.3, rng, d_x=c), want)


def test_refusals():
    x, rng = torch.zeros(4, 64, device="cuda"), rng_of(0, 0)
    for bad in (dict(rng=None), dict(rng=rng.int()), dict(x=x.half()), dict(residual=x[:2]), dict(y=x.bfloat16()),
                dict(x=torch.zeros(4, 128, device="cuda")[:, ::2]), dict(x=torch.zeros((), device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_dropout(**(dict(x=x, p=0.5, rng=rng) | bad))
    wide = torch.zeros(4 * 64 + 8, device="cuda")
    for bad in (dict(p=1.0), dict(p=-0.5), dict(p=float("nan")), dict(x=wide[:256].view(4, 64), y=wide[8:264].view(4, 64)),
                dict(x=torch.zeros(0, 64, device="cuda"))):
        with pytest.raises(T.TTTError):
            T.ttt_forward_dropout(**(dict(x=x, p=0.5, rng=rng) | bad))


def test_replayed():
    x, rng = torch.randn(100, 384, device="cuda"), rng_of(1, 2)
    y, z = torch.empty_like(x), torch.empty_like(x)

    def call():
        T.ttt_forward_dropout(x, 0.5, rng, y=y)
        T.ttt_backward_dropout(y, 0.5, rng, d_x=z)

    replays(call, [y, z], lambda: T.ttt_forward_dropout(x, 0.1, rng))


def test_rows_past_32_bits():
    """More than 2^32 elements, bf16: the last rows are those of a call on them alone, at their counters."""
    C, M = 1 << 12, (1 << 20) + 3
    x = torch.ones(M, C, device="cuda", dtype=torch.bfloat16)
    rng = rng_of(9, 0)
    y = T.ttt_forward_dropout(x, 0.5, rng, y=x)[-5:].clone()
    del x
    rng[1] += (M - 5) * (C // 8)
    assert torch.equal(y, T.ttt_forward_dropout(torch.ones(5, C, device="cuda", dtype=torch.bfloat16), 0.5, rng))
