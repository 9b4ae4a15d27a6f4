"""Shared pieces of the block operators' GPU tests: seeded inputs of either I/O type and the bound that
outputs are held to.

The bound. An output of type t is rounded once, by at most u_t = finfo(t).eps / 2 of its value (2^-8 of
bf16, 2^-24 of fp32). Before that everything is fp32, where each rounding is at most u = 2^-24 of an
intermediate, and an operator's intermediates add up to at most some c of them at the output's largest
magnitude: |got - ref| <= u_t |ref| + c u max|ref|. c is set per operator from its arithmetic:
  C_NORM   sums of at most 64 values in a lane and 8 levels over lanes (72 u) in the mean and, again, in the
           variance, against inputs whose mean is up to a few deviations: 72 * 2 * 8 < 2048;
  C_CONV   4 products, a sigmoid (exp2, a reciprocal: a few u) and its argument's error: 256;
  C_SCAN   exp(dt A) is off by (2 |dt A| + 2) u plus dt's own 4 u |dt A|, and an error of the decay is
           kept for as long as the state is: 1 / (1 - exp(-dt |A|)) tokens. Steps are at least 0.01 and
           |A| at least 0.5, so 200 tokens at about 4 u, and the sums over states on top: 2048;
  C_SUM    gradients of parameters: sums over R <= 5000 rows of random sign in fixed-order partial sums of
           up to 64 + 64 + 16 terms, whose absolute sum is about sqrt(R) ~ 64 times the result: 144 * 64
           < 16384, where the terms themselves are an operator's outputs.
"""
import numpy as np
import torch

U = 2.0 ** -24
C_NORM, C_CONV, C_SCAN, C_SUM = 2048, 256, 2048, 16384
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


class Inputs:
    """Seeded device tensors; f64() gives the same values on the host."""

    def __init__(self, seed, dtype):
        self.gen = torch.Generator().manual_seed(seed)
        self.io = DT[dtype]

    def normal(self, *shape, scale=1.0, mean=0.0, dtype=None):
        x = torch.randn(*shape, generator=self.gen) * scale + mean
        return x.to(self.io if dtype is None else dtype).cuda()

    def param(self, *shape, scale=1.0, mean=0.0):
        return self.normal(*shape, scale=scale, mean=mean, dtype=torch.float32)


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def check(name, got, ref, c):
    """got (device tensor) against ref (float64) to the bound above."""
    out = got.dtype
    got, ref = f64(got), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bound = torch.finfo(out).eps / 2 * np.abs(ref) + c * U * np.abs(ref).max(initial=0.0) + 1e-38
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{name}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    worst = float((off / bound).max(initial=0.0))
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound at {np.unravel_index((off / bound).argmax(), off.shape)}"


def sliced(t, lead, extra=5):
    """t's values in a slice of wider rows: the last `t.dim() - lead` dims are one row, `extra` elements are
    put before and behind it (filled with NaN)."""
    width = int(np.prod(t.shape[lead:]))
    rows = torch.full((*t.shape[:lead], width + 2 * extra), float("nan"), dtype=t.dtype, device=t.device)
    rows[..., extra:extra + width] = t.reshape(*t.shape[:lead], width)
    return rows[..., extra:extra + width].unflatten(-1, t.shape[lead:])


def replays(fn, outs, between):
    """Captures fn into a graph (after one eager call), then replays it three times with eager work and a
    synchronisation between, the outputs overwritten before each; every replay must give the eager bits."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        between()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
