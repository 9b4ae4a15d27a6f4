"""RMS norm where its numbers end: rows of zeros and of numbers next to zero under a small eps or none, weights near the ends of
fp32, quotients next to halfway points of e4m3 with every kind of neighbour, and rows at any alignment bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
from lm_helpers import EPS, within  # noqa: E402
from seq_helpers import Inputs  # noqa: E402
from seq_reference import held  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

DEPTH = 24 + 6 + 16  # additions of a row's sum: in a lane, over lanes, over waves
LEAST = 2.0 ** -100 / 448


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
