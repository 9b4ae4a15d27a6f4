"""Shared pieces of the residual block's GPU tests."""
import torch

from oracle import lm_oracle as O

EPS = 1e-5


def rng_of(seed, offset):
    """rng of a call, from numbers below 2^64."""
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda")


def factors(seed, offset, p, M, C):
    return torch.from_numpy(O.factors(seed, offset, p, M, C)).cuda()


def within(name, got, ref):
    """got's values to ref = (value, bound), got's own rounding included in the bound already."""
    value, bound = ref
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    share = (got.double() - value).abs() / (bound + 1e-37)
    worst = float(share.max())
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound at {int(share.argmax())} of {tuple(got.shape)}"
