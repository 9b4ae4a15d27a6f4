"""The block operators on small whole numbers, where fp32 is exact in any order of sums (asserted: the terms' absolute values
add up to less than 2^24): outputs are the formulas' to the bit, so that no term of a walk, a segment or a partial sum can be
missing, doubled or misplaced. Sizes of several turns and many segments (seq_plans.py)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import seq_reference as R  # noqa: E402
from seq_helpers import DT  # noqa: E402
from seq_plans import CONV_CASES, NORM_CASES, SCAN_CASES  # noqa: E402

import test_sequence_layers_amd as T  # noqa: E402

LIMIT = 2.0 ** 24
ids = lambda c: "-".join(str(v) for v in c if not isinstance(v, (dict, list)))  # noqa: E731


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


class Whole:
    def __init__(self, seed, dtype):
        self.gen, self.io = torch.Generator(device="cuda").manual_seed(seed), DT[dtype]

    def __call__(self, *shape, share=1.0, low=-1, high=1, dtype=None):
        """Whole numbers from low to high, a share of them other than zero."""
        x = torch.randint(low, high + 1, shape, device="cuda", generator=self.gen).float()
        if share < 1:
            x = x * (torch.rand(*shape, device="cuda", generator=self.gen) < share)
        return x.to(dtype or self.io)

    def param(self, *shape, **k):
        return self(*shape, dtype=torch.float32, **k)


def same(name, got, value):
    assert float(value.abs().max()) < LIMIT, name
    assert got.shape == value.shape and torch.equal(got, value.to(got.dtype)), \
        f"{name}: {int((got != value.to(got.dtype)).sum())} of {value.numel()} entries differ"


@pytest.mark.parametrize("case", NORM_CASES, ids=ids)
def test_layernorm_gradient_sums(case):
    """d_bias of any width; d_weight and d_x where a row is half ones and half their opposites: its mean is 0 and
    its variance 1, of a power of two of channels without any rounding."""
    M, H, D, dtype = case[:4]
    print(f"layernorm M={M} H={H} D={D} {dtype}", flush=True)
    whole = Whole(M + D, dtype)
    shape = (M, H, D) if H > 1 else (M, D)
    d_y, w = whole(*shape, low=-2, high=2), whole.param(*shape[1:], low=1, high=2)
    x = torch.ones(shape, device="cuda")
    x[..., D // 2:] = -1.0
    x = x.gather(-1, torch.rand(*shape, device="cuda", generator=whole.gen).argsort(-1)).to(whole.io)
    d_x, d_weight, d_bias = T.ttt_backward_layernorm(x, w, d_y, 0.0)
    assert 2 * M < LIMIT
    same("d_bias", d_bias, d_y.double().sum(0))
    if D & (D - 1) == 0:
        xhat, g = x.double(), d_y.double() * w.double()
        same("d_weight", d_weight, (d_y.double() * xhat).sum(0))
        want = g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)
        same("d_x", d_x, want)  # (a multiple of 2^-14 below 16)
        same("y", T.ttt_forward_layernorm(x, w, None, 0.0), xhat * w.double())


@pytest.mark.parametrize("case", CONV_CASES, ids=ids)
def test_conv1d(case):
    B, N, C, K, dtype, _, state, lengths = case
    print(f"conv1d B={B} N={N} C={C} K={K} {dtype}", flush=True)
    whole = Whole(N + C, dtype)
    x, d_y, w, b = whole(B, N, C, low=-3, high=3), whole(B, N, C, low=-3, high=3), whole.param(C, K, low=-2, high=2), whole.param(C)
    s = whole(B, K - 1, C, low=-3, high=3) if state else None
    more = dict(state=s, lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert 9 * B * N < LIMIT
    ref = R.conv1d(x, w, b, d_y, **more)
    same("y", T.ttt_forward_conv1d(x, w, b, **more), ref["y"][0])
    for name, got in zip(("d_x", "d_weight", "d_bias", "d_state"), T.ttt_backward_conv1d(x, w, b, d_y, **more)):
        if got is not None:
            same(name, got, ref[name][0])


@pytest.mark.parametrize("case", SCAN_CASES, ids=ids)
def test_scan(case):
    """Steps of 0 and 1 (no softplus), A of 0: decays are 1, and states are sums of all tokens before. What the sums' terms
    add up to in absolute value (Q, H of the reference) is bounded by a run on the absolute values."""
    B, N, C, S, G, dtype, opt = case[:7]
    print(f"scan B={B} N={N} C={C} S={S} G={G} {dtype}", flush=True)
    whole = Whole(N + C + S, dtype)
    few = min(1.0, 24 / N)
    s = dict(u=whole(B, N, C), delta=whole(B, N, C, low=0, share=few), A=torch.zeros(C, S, device="cuda"), Bm=whole(B, N, G, S),
             Cm=whole(B, N, G, S), D=whole.param(C), h0=whole.param(B, C, S), softplus=False)
    lengths = opt.get("lengths")
    s["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    d_y = whole(B, N, C, share=few)
    most = R.scan(**{k: v.abs() if torch.is_tensor(v) and k != "lengths" else v for k, v in s.items()}, d_y=d_y.abs())
    assert all(float(v.max()) < LIMIT for v, _ in most.values())
    del most
    end = torch.empty(B, C, S, device="cuda")
    y = T.ttt_forward_selective_scan(**s, h_out=end)
    ref = R.scan(**s)
    same("y", y, ref["y"][0])
    same("h_out", end, ref["h_out"][0])
    names = ("d_u", "d_delta", "d_A", "d_B", "d_C", "d_D", "d_delta_bias", "d_z", "d_h0")
    got = dict(zip(names, T.ttt_backward_selective_scan(**s, d_y=d_y)))
    ref = R.scan(**s, d_y=d_y)
    for name in names:
        if got[name] is not None:
            same(name, got[name], ref[name][0])
