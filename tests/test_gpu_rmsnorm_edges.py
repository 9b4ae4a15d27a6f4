"""RMS norm where its numbers end: rows of zeros and of numbers next to zero under a small eps or none, weights near the ends of
fp32, quotients next to halfway points of e4m3 with every kind of neighbour, and rows at any alignment bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
from lm_helpers import within  # noqa: E402
from seq_helpers import Inputs  # noqa: E402
from seq_reference import held  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

DEPTH = 24 + 6 + 16  # additions of a row's sum: in a lane, over lanes, over waves


def _within(got, ref, group, D):
    """An 8-bit output and its scales to the bounds."""
    q, scales = got
    within("scales", scales, (ref["scales"][0], ref["scales"][1] + 1e-40))
    within("y * scales", (q.double().unflatten(-1, (-1, group or D)) * scales.double()[..., None]).flatten(-2), ref["deq"])


# --------------------------------------------------------------------------- zeros and next to zero
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
