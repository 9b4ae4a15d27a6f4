"""RMS norm where its numbers end: rows of zeros and of numbers next to zero under a small eps or none, weights near the ends of
fp32, quotients next to halfway points of e4m3 with every kind of neighbour, and rows at any alignment bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
from lm_helpers import EPS, rng_of, within  # noqa: E402
from seq_helpers import Inputs, sliced  # noqa: E402
from seq_reference import held  # noqa: E402

from oracle import lm_oracle as O  # noqa: E402
import test_sequence_layers_amd as T  # noqa: E402

DEPTH = 24 + 6 + 16  # additions of a row's sum: in a lane, over lanes, over waves
LEAST = 2.0 ** -100 / 448


def _bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def _within(got, ref, group, D):
    """An 8-bit output and its scales to the bounds."""
    q, scales = got
    within("scales", scales, (ref["scales"][0], ref["scales"][1] + 1e-40))
    within("y * scales", (q.double().unflatten(-1, (-1, group or D)) * scales.double()[..., None]).flatten(-2), ref["deq"])


# --------------------------------------------------------------------------- zeros and next to zero
@pytest.mark.parametrize("eps", [2.0 ** -40, 2.0 ** -100, 2.0 ** -126])
@pytest.mark.parametrize("D,group,dtype", [(64, 0, "bf16"), (96, 32, "fp32"), (256, 128, "bf16"), (1001, 0, "fp32"), (4096, 64, "bf16")])
def test_rows_and_groups_of_zeros_in_8_bits(D, group, dtype, eps):
    """Zeros, at the least scale, whatever eps is: padding's rows, and groups that their weights or their row leave without a value."""
    i = Inputs(D, dtype)
    x, w = i.normal(9, D), i.param(D, mean=1.0, scale=0.2)
    x[[0, 3, 8]] = 0
    size = group or D
    if group:
        x[1:3, size:2 * size] = 0
        w[:size] = 0
    y, scales = T.ttt_forward_rmsnorm_e4m3(x, w, eps, group=group)
    empty = torch.zeros_like(scales, dtype=torch.bool)
    empty[[0, 3, 8]] = True
    if group:
        empty[1:3, 1] = True
        empty[:, 0] = True
    wide = empty.repeat_interleave(size, -1)
    assert not y.float()[wide].any() and bool((y.float()[~wide] != 0).any())
    assert float((scales.double()[empty] / LEAST - 1).abs().max()) < 2.0 ** -23
    _within((y, scales), R.rmsnorm_e4m3(x, w, eps, DEPTH, size), group, D)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_group_of_zeros_in_a_row_next_to_zero(dtype):
    """No eps, rows of 1e-7 and of 1e-15, and a group of zeros in them."""
    i = Inputs(5, dtype)
    x, w = i.normal(8, 256), i.param(256, mean=1.0, scale=0.2)
    x *= torch.tensor([1e-7, 1e-15], device="cuda").repeat(4)[:, None].to(x.dtype)
    x[:, 32:64] = 0
    y, scales = T.ttt_forward_rmsnorm_e4m3(x, w, 0.0, group=32)
    assert not y.float()[:, 32:64].any() and float((scales.double()[:, 1] / LEAST - 1).abs().max()) < 2.0 ** -23
    _within((y, scales), R.rmsnorm_e4m3(x, w, 0.0, DEPTH, 32), 32, 256)


def test_outputs_below_the_least_scale():
    """Groups whose largest output is below 2^-100 take that as their largest: 1e-38 under eps 2^-40 comes to 1e-32."""
    i = Inputs(6, "fp32")
    x, w = (i.normal(8, 256).double() * 1e-38).float(), i.param(256, mean=1.0, scale=0.2)
    got = T.ttt_forward_rmsnorm_e4m3(x, w, 2.0 ** -40, group=64)
    assert float((got[1].double() / LEAST - 1).abs().max()) < 2.0 ** -23 and bool(got[0].float().any())
    _within(got, R.rmsnorm_e4m3(x, w, 2.0 ** -40, DEPTH, 64), 64, 256)


@pytest.mark.parametrize("size", [-45, -60, -74, -80, -100, -126, -132])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (768, "fp32"), (1001, "bf16"), (1001, "fp32"), (4096, "bf16"), (16384, "fp32")])
def test_rows_next_to_zero_are_normed_like_others(D, dtype, size):
    """Squares below fp32's smallest numbers, with no eps and with one of their size: y and back, and in 8 bits."""
    i = Inputs(D, dtype)
    x, w, d_y, d_sum = i.normal(5, D), i.param(D, mean=1.0, scale=0.2), i.normal(5, D, scale=2.0 ** -20), i.normal(5, D)
    x = (x.double() * 2.0 ** size).to(x.dtype)
    x[3] = Inputs(7, dtype).normal(D)  # an ordinary row among them
    for eps in (0.0, 2.0 ** (2 * size) if size > -74 else 2.0 ** -149):
        held("y", T.ttt_forward_rmsnorm(x, w, eps), R.rmsnorm(x, w, eps, DEPTH)["y"])
        d_s, _, d_w = T.ttt_backward_rmsnorm(x, w, d_y, eps, d_sum=d_sum)
        ref = R.rmsnorm_backward(x, w, d_y, eps, DEPTH, 140, d_sum)
        held("d_s", d_s, ref["d_s"])
        held("d_weight", d_w, ref["d_weight"])
        _within(T.ttt_forward_rmsnorm_e4m3(x, w, eps), R.rmsnorm_e4m3(x, w, eps, DEPTH, D), 0, D)


def test_a_gradient_of_nothing_stays_nothing():
    """Rows so near to zero that 1 / rms is past fp32: a d_y of zeros gives zeros, and what arrives at the sum passes through."""
    i = Inputs(8, "fp32")
    x = (i.normal(4, 96).double() * 2.0 ** -138).float()
    d_sum = i.normal(4, 96)
    d_s, _, d_w = T.ttt_backward_rmsnorm(x, i.param(96), torch.zeros_like(x), 0.0, d_sum=d_sum)
    assert torch.equal(d_s, d_sum) and not d_w.any()


@pytest.mark.parametrize("group", [0, 64])
def test_weights_and_rows_at_the_ends_of_fp32_in_8_bits(group):
    """The product of a row and its weights is past fp32 or next to nothing before the norm, and ordinary behind it."""
    i = Inputs(9, "fp32")
    x, w = i.normal(6, 512), i.param(512, mean=1.0, scale=0.2)
    for row, weight, eps in ((1e3, 1e36, EPS), (1e-42, 1.0, 2.0 ** -100), (1e18, 1e30, EPS), (1e-20, 1e-25, 2.0 ** -149), (1e-3, 1e-28, EPS)):
        a, b = (x.double() * row).float(), (w.double() * weight).float()
        _within(T.ttt_forward_rmsnorm_e4m3(a, b, eps, group=group), R.rmsnorm_e4m3(a, b, eps, DEPTH, group or 512), group, 512)


def test_infinities_and_nan_in_groups():
    """A group whose output has a NaN is NaN, one whose output has an infinity is NaN there and zeros elsewhere; an infinite entry of a row is a
    NaN of the output and leaves the row's other groups zeros, a NaN leaves nothing."""
    i = Inputs(10, "fp32")
    x, w = i.normal(5, 256), i.param(256, mean=1.0, scale=0.2)
    w[200] = float("inf")
    x[1, 70], x[2, 5] = -float("inf"), float("nan")
    want = R.rmsnorm_e4m3(x, w.clamp(max=9), EPS, DEPTH, 64)
    y, scales = T.ttt_forward_rmsnorm_e4m3(x, w, EPS, group=64)
    y = y.double().view(5, 4, 64)
    for m in (0, 3, 4):
        assert torch.isnan(y[m, 3, 8]) and not y[m, 3, :8].any() and not y[m, 3, 9:].any() and scales[m, 3] == float("inf")
        within("y * scales", (y[m, :3] * scales[m, :3, None].double()).flatten(), tuple(t[m, :192] for t in want["deq"]))
    assert torch.isnan(y[1, 1]).all() and torch.isnan(scales[1, 1]) and not y[1, [0, 2]].any()
    assert torch.isnan(y[2]).all() and torch.isnan(scales[2]).all()


# --------------------------------------------------------------------- next to halfway points of e4m3
def _beside(ties, rows, D, group, seed=0, top=None):
    """Rows [rows, D] of fp32 whose groups each hold their largest, `top` of the row, and numbers next to (at most 2^-24 of themselves
    from) halfway points of that group's scale, and their quotients by it in float64 (weights of one leave them so)."""
    gen = torch.Generator().manual_seed(seed)
    if top is None:
        top = (torch.rand(rows, 1, generator=gen) + 1) * 2.0 ** torch.arange(rows)[:, None].remainder(40).sub(20).float()
    n = rows * D // group
    v = ties[torch.randint(0, len(ties), (n, group), generator=gen)] * (torch.randint(0, 2, (n, group), generator=gen) * 2 - 1)
    v[torch.arange(n), torch.randint(0, group, (n,), generator=gen)] = 448.0
    x = (v.view(rows, D) * top.double() / 448).float()
    return x, x.double() * 448 / top.double()


NORMAL = torch.tensor([(8.5 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)], dtype=torch.float64)
NORMAL = NORMAL[NORMAL < 448]
SMALL = (torch.arange(8, dtype=torch.float64) + 0.5) * 2.0 ** -9


def _to_e4m3(q):
    return torch.from_numpy(O.e4m3(q.numpy()))


@pytest.mark.parametrize("D,group", [(96, 32), (160, 32), (384, 128), (384, 64), (768, 128), (1312, 32), (2592, 32), (64, 64), (16000, 128)])
def test_halfway_points_beside_lanes_without_a_value(D, group):
    """Widths that leave lanes of a row's last access empty: every value is the nearest of its quotient in 64 bits."""
    x, q = _beside(NORMAL, 64, D, group, D)
    y, _ = T.ttt_forward_rmsnorm_e4m3(x.cuda(), torch.ones(D, device="cuda"), EPS, group=group)
    assert torch.equal(y.double().cpu(), _to_e4m3(q))


@pytest.mark.parametrize("D,group", [(32, 32), (64, 32), (128, 128), (128, 64), (256, 64), (20, 20)])
@pytest.mark.parametrize("ties", [NORMAL, SMALL], ids=["normal", "small"])
def test_a_row_in_8_bits_is_its_own_whatever_its_neighbours(D, group, ties):
    """Rows that share a wave with zeros, infinities and NaN: the bits of the rows by themselves, and the nearest."""
    x, q = _beside(ties, 48, D, group, D)
    w = torch.ones(D, device="cuda")
    alone = T.ttt_forward_rmsnorm_e4m3(x.cuda(), w, EPS, group=0 if group == D else group)
    assert torch.equal(alone[0].double().cpu(), _to_e4m3(q))
    for bad in (0.0, float("nan"), float("inf"), 1e-44):
        both = torch.full((96, D), bad)
        both[1::2] = x
        got = T.ttt_forward_rmsnorm_e4m3(both.cuda(), w, EPS, group=0 if group == D else group)
        for a, b in zip(got, alone):
            assert torch.equal(_bits(a[1::2]), _bits(b)), bad


@pytest.mark.parametrize("D,group", [(128, 128), (384, 128), (512, 32), (1001, 1001), (8192, 64)])
def test_halfway_points_below_the_normal_numbers(D, group):
    """Below 2^-6 of the scale, where e4m3's steps stay 2^-9: the nearest there too, and of exact halves the even one."""
    x, q = _beside(SMALL, 64, D, group, D)
    whole = 0 if group == D else group
    y, _ = T.ttt_forward_rmsnorm_e4m3(x.cuda(), torch.ones(D, device="cuda"), EPS, group=whole)
    assert torch.equal(y.double().cpu(), _to_e4m3(q))
    x, q = _beside(torch.cat([SMALL, NORMAL]), 64, D, group, D + 1, torch.full((64, 1), 448.0))
    y, _ = T.ttt_forward_rmsnorm_e4m3(x.cuda(), torch.ones(D, device="cuda"), EPS, group=whole)
    assert torch.equal(x.double(), q) and torch.equal(y.double().cpu(), _to_e4m3(q))


# ------------------------------------------------------------------------------------- alignment
@pytest.mark.parametrize("D,dtype", [(512, "bf16"), (1001, "bf16"), (768, "fp32"), (65, "fp32"), (4096, "bf16")])
def test_rows_at_any_alignment_give_the_same_bits(D, dtype):
    i = Inputs(13, dtype)
    x, w, res, d_y, d_sum = i.normal(50, D), i.param(D), i.normal(50, D), i.normal(50, D), i.normal(50, D)
    rng = rng_of(1 << 63, 9)
    want = (*T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=0.25, rng=rng), *T.ttt_forward_rmsnorm_e4m3(x, w, EPS),
            *T.ttt_backward_rmsnorm(x, w, d_y, EPS, d_sum=d_sum, p=0.25, rng=rng))
    for extra in (1, 2, 3, 4, 8):
        a = sliced(x, 1, extra)
        got = (*T.ttt_forward_rmsnorm(a, w, EPS, residual=res, p=0.25, rng=rng), *T.ttt_forward_rmsnorm_e4m3(a, w, EPS),
               *T.ttt_backward_rmsnorm(a, w, d_y, EPS, d_sum=d_sum, p=0.25, rng=rng))
        assert len(got) == len(want) and all(torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want)), extra
