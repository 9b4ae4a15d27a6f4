"""RMS norm with the residual's addition, dropout and an output in 8 bits, forward and backward, against float64 within what
fp32 can lose, entry by entry (lm_reference.py). A row's sums: at most 24 elements in a lane, 6 levels over lanes, 16 waves."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lm_reference as R  # noqa: E402
from lm_helpers import EPS, factors, rng_of, within  # noqa: E402
from seq_helpers import Inputs, replays, sliced  # noqa: E402
from seq_reference import held  # noqa: E402

from oracle import lm_oracle as O  # noqa: E402
import test_sequence_layers_amd as T  # noqa: E402

DEPTH = 24 + 6 + 16
DT = {"bf16": T.TTT_BF16, "fp32": T.TTT_F32}
CASES = [  # M, H, D, dtype, sliced
    (1, 1, 1, "fp32", False), (3, 1, 7, "bf16", False), (5, 1, 33, "fp32", True), (257, 1, 65, "bf16", False),
    (9, 12, 64, "bf16", False), (130, 12, 64, "bf16", True), (77, 3, 64, "fp32", False), (33, 5, 16, "bf16", False),
    (17, 2, 32, "fp32", True), (6, 7, 24, "bf16", True), (21, 3, 10, "fp32", False), (100, 1, 100, "bf16", False),
    (64, 1, 384, "bf16", True), (1, 1, 768, "bf16", False), (35, 1, 768, "fp32", True), (300, 1, 1001, "fp32", False),
    (41, 1, 1001, "bf16", True), (23, 1, 1280, "bf16", False), (10, 1, 2056, "bf16", False), (7, 1, 2050, "fp32", False),
    (12, 1, 4096, "fp32", False), (5, 2, 4100, "bf16", False), (9, 1, 8192, "bf16", True), (3, 1, 16384, "fp32", False),
    (3, 1, 16383, "bf16", False), (2, 1, 16384, "bf16", False), (5000, 1, 8, "fp32", False), (4100, 1, 128, "bf16", False),
    (3, 300, 8, "fp32", False), (12544, 1, 384, "bf16", False), (1537, 1, 1001, "fp32", False), (5003, 1, 768, "bf16", True),
]
ids = lambda c: "-".join(str(v) for v in c)  # noqa: E731


def _inputs(M, H, D, dtype, cut):
    i = Inputs(M + 7 * D, dtype)
    shape = (M, H, D) if H > 1 else (M, D)
    x, w = i.normal(*shape, mean=0.5), i.param(*shape[1:], scale=0.2, mean=1.0)
    # an extra of 8 elements keeps a slice's rows on 16 bytes, of 5 does not
    return i, shape, sliced(x, 1, 8 if D % 16 == 0 else 5) if cut else x, w


def _rows_depth(M, H, D, dtype):
    """A parameter's sums: a group's turns (there are no fewer groups than workgroups), at most 128 groups of a workgroup, the
    partial rows 64 at a time and 6 levels."""
    rows = T.load_library().ttt_backward_rmsnorm_workspace(DT[dtype], M, H, D) // (4 * H * D)
    return M // max(1, rows // 2) + 1 + 128 + rows // 64 + 7


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_norm(case):
    M, H, D, dtype, cut = case
    print(f"rmsnorm M={M} H={H} D={D} {dtype} sliced={cut}", flush=True)
    i, shape, x, w = _inputs(*case)
    d_y = i.normal(*shape)
    held("y", T.ttt_forward_rmsnorm(x, w, EPS), R.rmsnorm(x, w, EPS, DEPTH)["y"])
    d_s, d_x, d_w = T.ttt_backward_rmsnorm(x, w, d_y, EPS)
    assert d_x is None
    ref = R.rmsnorm_backward(x, w, d_y, EPS, DEPTH, _rows_depth(M, H, D, dtype))
    held("d_s", d_s, ref["d_s"])
    held("d_weight", d_w, ref["d_weight"])


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] == 1], ids=ids)
def test_residual_and_dropout(case, p):
    """The sum, its norm, and back, with the gradient that arrives at the sum."""
    M, H, D, dtype, cut = case
    print(f"rmsnorm with residual M={M} D={D} {dtype} sliced={cut} p={p}", flush=True)
    i, shape, x, w = _inputs(*case)
    res, d_y, d_sum = i.normal(*shape, scale=2.0), i.normal(*shape), i.normal(*shape)
    rng, f = (rng_of(12345, (1 << 33) + 7), factors(12345, (1 << 33) + 7, p, M, D)) if p else (None, None)
    y, s = T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=p, rng=rng)
    ref = R.rmsnorm(x, w, EPS, DEPTH, res, f)
    held("y", y, ref["y"])
    held("sum", s, ref["sum"])
    d_s, d_x, d_w = T.ttt_backward_rmsnorm(s, w, d_y, EPS, d_sum=d_sum, p=p, rng=rng)
    ref = R.rmsnorm_backward(s, w, d_y, EPS, DEPTH, _rows_depth(M, H, D, dtype), d_sum, f)
    held("d_s", d_s, ref["d_s"])
    held("d_weight", d_w, ref["d_weight"])
    if p:
        held("d_x", d_x, ref["d_x"])
        assert torch.equal(d_x != 0, (f > 0) & (d_x != 0)) and float(((f > 0) & (d_x == 0)).double().mean()) < 0.01
    else:
        assert d_x is None


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_narrow_width_at_every_alignment(dtype):
    """Widths of 1 .. 40 and around whole accesses, rows starting at every element of 16 bytes: the sums of a row to the bounds, and
    what is around the outputs as it was."""
    for D in [*range(1, 41), 63, 65, 127, 129, 511, 513, 1023, 1025, 2047, 2049]:
        i = Inputs(D, dtype)
        e = D % 8
        w, x, res, d_y = i.param(D, mean=1.0, scale=0.2), sliced(i.normal(5, D), 1, e), i.normal(5, D), i.normal(5, D)

        def inside():
            around = torch.full((5 * D + 32,), 7.0, dtype=i.io, device="cuda")
            return around, around[8 + e:8 + e + 5 * D].view(5, D)

        (by, y), (bs, s), (bd, d_s) = inside(), inside(), inside()
        T.ttt_forward_rmsnorm(x, w, EPS, residual=res, y=y, sum_out=s)
        ref = R.rmsnorm(x, w, EPS, DEPTH, res)
        held(f"y of {D}", y, ref["y"])
        held(f"sum of {D}", s, ref["sum"])
        d_w = T.ttt_backward_rmsnorm(s, w, d_y, EPS, d_s=d_s)[2]
        ref = R.rmsnorm_backward(s, w, d_y, EPS, DEPTH, 140)
        held(f"d_s of {D}", d_s, ref["d_s"])
        held(f"d_weight of {D}", d_w, ref["d_weight"])
        for around in (by, bs, bd):
            assert bool((around[:8 + e] == 7).all()) and bool((around[8 + e + 5 * D:] == 7).all())
        q, scales = T.ttt_forward_rmsnorm_e4m3(x, w, EPS)
        ref = R.rmsnorm_e4m3(x, w, EPS, DEPTH, D)
        within(f"y * scales of {D}", q.double() * scales.double(), ref["deq"])


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,H,D,dtype,group,cut", [
    (1, 1, 1, "fp32", 0, False), (3, 1, 7, "bf16", 0, False), (16, 1, 768, "bf16", 0, False), (5, 1, 33, "fp32", 0, True),
    (9, 12, 64, "bf16", 0, False), (9, 12, 64, "bf16", 32, True), (33, 5, 32, "fp32", 32, False), (77, 3, 128, "fp32", 64, False),
    (130, 1, 384, "bf16", 128, False), (130, 1, 1536, "bf16", 128, False), (35, 1, 768, "fp32", 128, True), (300, 1, 1001, "fp32", 0, False),
    (23, 1, 1280, "bf16", 64, False), (10, 1, 2048, "bf16", 32, False), (12, 1, 4096, "fp32", 128, False), (5, 1, 8192, "bf16", 128, False),
    (3, 1, 16384, "fp32", 0, False), (2, 1, 16384, "bf16", 64, False), (3, 1, 16383, "bf16", 0, False), (7, 1, 96, "bf16", 32, False),
    (700, 1, 160, "fp32", 32, False)])
def test_e4m3(M, H, D, dtype, group, cut, add):
    if add and H > 1:
        pytest.skip("a residual needs H = 1")
    print(f"rmsnorm e4m3 M={M} H={H} D={D} {dtype} group={group} sliced={cut} residual={add}", flush=True)
    i, shape, x, w = _inputs(M, H, D, dtype, cut)
    res = i.normal(*shape, scale=2.0) if add else None
    got = T.ttt_forward_rmsnorm_e4m3(x, w, EPS, residual=res, group=group)
    assert len(got) == 2 + add and got[0].dtype == torch.float8_e4m3fn
    ref = R.rmsnorm_e4m3(x, w, EPS, DEPTH, group or D, res)
    within("scales", got[1], (ref["scales"][0], ref["scales"][1] + 1e-40))
    q = got[0].double().unflatten(-1, (-1, group or D))
    within("y * scales", (q * got[1].double()[..., None]).flatten(-2), ref["deq"])
    assert bool((q.abs().amax(-1) == 448).all())  # a group's largest
    if add:
        held("sum", got[2], ref["sum"])


def test_e4m3_rounds_to_the_nearest():
    """A row of every number and every tie between two, its weight its own root mean square: the norm is the row again."""
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    table = table[torch.isfinite(table)].sort().values
    v = torch.cat([table, (table[1:] + table[:-1]) / 2]).double()
    v = torch.cat([v, torch.zeros(512 - v.numel())]).cuda()
    x = v.float()[None].expand(3, -1).contiguous()
    rms = float((v * v).mean().sqrt())
    w = torch.full((512,), rms, device="cuda", dtype=torch.float64).float()
    y, scales = T.ttt_forward_rmsnorm_e4m3(x, w, 0.0)
    # the norm's output is off by a few 2^-24 of it, so ties may fall either way, and all else is itself
    got = y[0].double().cpu()
    want = v.cpu()
    n = table.numel()
    assert torch.equal(got[:n], want[:n]) and float((scales - 1).abs().max()) < 2e-6
    below, above = table[:-1].double(), table[1:].double()
    mid = got[n:2 * n - 1]
    assert bool(((mid == below) | (mid == above)).all())


@pytest.mark.parametrize("D,group", [(128, 0), (256, 128), (4096, 0)])
def test_e4m3_takes_values_beside_a_tie_to_their_own_side(D, group):
    """Numbers of fp32 next to halfway points of their group's scale, off by at most 2^-24 of themselves: with weights of one the
    quotient by the group's largest is exact before it is rounded to 8 bits, and the nearest is the quotient's in 64 bits."""
    ties = torch.tensor([(8.5 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)], dtype=torch.float64)
    ties = ties[ties < 448]
    i = Inputs(D, "fp32")
    top = (i.normal(64, 1).abs().clamp(min=0.01) * 2.0 ** torch.arange(-20, 44, device="cuda")[:, None].float()).cpu()
    v = torch.zeros(64, D, dtype=torch.float64)
    v[:, 0] = 448
    v[:, 1:1 + len(ties)] = ties
    if group:
        v[:, group:] = -v[:, :-group]
    if D > 512:
        v = v.roll(1000, 1)
    x = (v * top.double() / 448).float()
    q = x.double() * 448 / top.double()
    y, scales = T.ttt_forward_rmsnorm_e4m3(x.cuda(), torch.ones(D, device="cuda"), EPS, group=group)
    assert torch.equal(y.double().cpu(), torch.from_numpy(O.e4m3(q.numpy())))
    # a scale: half of what the squares' sum loses, two steps each of the mean, the root and its inverse, two products
    norm = x.double() / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt()
    assert float((scales.double().cpu() * 448 / norm.abs().amax(-1, keepdim=True) - 1).abs().max()) < (DEPTH / 2 + 10) * 2.0 ** -24


def test_in_place():
    i = Inputs(3, "bf16")
    x, res, w, d_y, d_sum = i.normal(70, 520), i.normal(70, 520), i.param(520), i.normal(70, 520), i.normal(70, 520)
    rng = rng_of(1, 2)
    y, s = T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=0.2, rng=rng)
    stream = res.clone()
    version = stream._version
    y2, s2 = T.ttt_forward_rmsnorm(x, w, EPS, residual=stream, p=0.2, rng=rng, sum_out=stream)
    assert s2 is stream and torch.equal(stream, s) and torch.equal(y, y2) and stream._version > version
    stream = res.clone()
    q = T.ttt_forward_rmsnorm_e4m3(x, w, EPS, residual=res)
    q2 = T.ttt_forward_rmsnorm_e4m3(x, w, EPS, residual=stream, sum_out=stream)
    assert q2[2] is stream and all(torch.equal(a.float(), b.float()) for a, b in zip(q, q2))
    want = T.ttt_backward_rmsnorm(s, w, d_y, EPS, d_sum=d_sum, p=0.2, rng=rng)
    got = T.ttt_backward_rmsnorm(s, w, d_y, EPS, d_sum=d_sum, p=0.2, rng=rng, d_s=d_sum)
    assert got[0] is d_sum and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 768, 1001, 4096])
def test_rows_of_large_and_of_small_numbers(dtype, D):
    """Squares past fp32's largest number, and rows of zeros: y to the bounds (eps is nothing, or all there is)."""
    i = Inputs(D, dtype)
    x, w = i.normal(6, D), i.param(D, scale=0.2, mean=1.0)
    x[1], x[3], x[4] = x[1] * 2.0 ** 100, x[3] * 2.0 ** 66, 0
    held("y", T.ttt_forward_rmsnorm(x, w, EPS), R.rmsnorm(x, w, EPS, DEPTH)["y"])
    d_y = i.normal(6, D)
    d_s, _, d_w = T.ttt_backward_rmsnorm(x, w, d_y, EPS)
    ref = R.rmsnorm_backward(x, w, d_y, EPS, DEPTH, 140)
    held("d_s", d_s, ref["d_s"])
    held("d_weight", d_w, ref["d_weight"])
    q, scales = T.ttt_forward_rmsnorm_e4m3(x, w, EPS)
    assert not q[4].float().any() and abs(float(scales[4]) / (2.0 ** -100 / 448) - 1) < 2.0 ** -23
    q, scales = T.ttt_forward_rmsnorm_e4m3(x, w, 0.0)
    assert bool(torch.isnan(q[4].float()).all()) and bool(torch.isfinite(q[[0, 1, 2, 3, 5]].float()).all())  # 0 / 0


@pytest.mark.parametrize("D", [256, 1001])
def test_rows_that_are_not_finite_stay_their_own(D):
    i = Inputs(12, "bf16")
    x, res, w = i.normal(6, D), i.normal(6, D), i.param(D)
    rng, f = rng_of(5, 5), factors(5, 5, 0.5, 6, D)
    want, s = T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=0.5, rng=rng)
    bad = x.clone()
    bad[f == 0] = float("nan")  # dropped: no part of the sum, whatever they are
    y, s2 = T.ttt_forward_rmsnorm(bad, w, EPS, residual=res, p=0.5, rng=rng)
    assert torch.equal(y, want) and torch.equal(s, s2)
    res[1, 3], res[4, D - 1] = float("inf"), float("nan")
    y, s2 = T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=0.5, rng=rng)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], want[keep]) and torch.isnan(y[4]).all()
    assert torch.isnan(y[1, 3]) and not y[1, :3].any() and not y[1, 4:].any()
    q, scales, _ = T.ttt_forward_rmsnorm_e4m3(x, w, EPS, residual=res)
    assert torch.isnan(scales[[1, 4]]).all() and torch.isnan(q[[1, 4]].float()).all() and torch.isfinite(q[keep].float()).all()


def test_aligned_and_unaligned_rows_agree():
    """The element-wise path against the 16-byte one on the same values, and the same mask."""
    i = Inputs(13, "bf16")
    x, w, res, d_y = i.normal(50, 512), i.param(512), i.normal(50, 512), i.normal(50, 512)
    off, rng = sliced(x, 1, 3), rng_of(1 << 63, 9)
    f = factors(1 << 63, 9, 0.25, 50, 512)
    ref = R.rmsnorm(x, w, EPS, DEPTH, res, f)
    for a in (x, off):
        y, s = T.ttt_forward_rmsnorm(a, w, EPS, residual=res, p=0.25, rng=rng)
        held("y", y, ref["y"])
        held("sum", s, ref["sum"])
    ref = R.rmsnorm_backward(x, w, d_y, EPS, DEPTH, 140, None, f)
    for a in (x, off):
        d_s, d_x, d_w = T.ttt_backward_rmsnorm(a, w, d_y, EPS, p=0.25, rng=rng)
        held("d_s", d_s, ref["d_s"])
        held("d_x", d_x, ref["d_x"])
        held("d_weight", d_w, ref["d_weight"])


def test_a_probability_of_less_than_half_a_step_drops_nothing():
    i = Inputs(14, "fp32")
    x, w, res, d_y = i.normal(5, 64), i.param(64), i.normal(5, 64), i.normal(5, 64)
    rng = rng_of(1, 1)
    y, s = T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=1e-6, rng=rng)
    assert torch.equal(s, x + res)
    d_s, d_x, _ = T.ttt_backward_rmsnorm(s, w, d_y, EPS, p=1e-6, rng=rng)
    assert torch.equal(d_s, d_x)


def test_rows_past_32_bits():
    """Rows whose stride takes them past 2^32 elements: the last row's results are those of a call on it alone."""
    D, stride = 777, 2_400_000_001
    rows = torch.zeros(2 * stride + D, device="cuda", dtype=torch.bfloat16)  # 9.6 GB
    x, i = rows.as_strided((3, D), (stride, 1)), Inputs(1, "bf16")
    x.copy_(i.normal(3, D))
    w, d_y = i.param(D, mean=1.0, scale=0.2), i.normal(3, D)
    y, d_s = T.ttt_forward_rmsnorm(x, w, EPS), T.ttt_backward_rmsnorm(x, w, d_y, EPS)[0]
    assert torch.equal(y[2:], T.ttt_forward_rmsnorm(x[2:].contiguous(), w, EPS))
    assert torch.equal(d_s[2:], T.ttt_backward_rmsnorm(x[2:].contiguous(), w, d_y[2:].contiguous(), EPS)[0])


def test_refusals():
    x, w, res = torch.zeros(4, 64, device="cuda"), torch.zeros(64, device="cuda"), torch.zeros(4, 64, device="cuda")
    rng = rng_of(0, 0)
    for bad in (dict(weight=w.double()), dict(weight=torch.zeros(32, device="cuda")), dict(x=x.half()),
                dict(residual=res.bfloat16()), dict(residual=res[:2]), dict(residual=res.t().contiguous().t()),
                dict(sum_out=res), dict(residual=res, p=0.5), dict(residual=res, p=0.5, rng=rng.int()),
                dict(residual=res, p=0.5, rng=rng.cpu()), dict(residual=res, p=0.5, rng=rng[:1])):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_forward_rmsnorm(**(dict(x=x, weight=w) | bad))
    for bad in (dict(eps=-1.0), dict(y=x), dict(p=0.5, rng=rng), dict(residual=res, p=1.0, rng=rng),
                dict(residual=res, p=-0.1, rng=rng), dict(residual=res, p=float("nan"), rng=rng), dict(residual=res, y=res),
                dict(residual=res, p=0.9999999, rng=rng), dict(residual=res, sum_out=x)):
        with pytest.raises(T.TTTError):
            T.ttt_forward_rmsnorm(**(dict(x=x, weight=w) | bad))
    heads = torch.zeros(4, 2, 32, device="cuda")
    with pytest.raises(T.TTTError):
        T.ttt_forward_rmsnorm(heads, torch.zeros(2, 32, device="cuda"), residual=torch.zeros_like(heads))
    for bad in (dict(group=48), dict(group=-1), dict(y=torch.zeros(4, 64, device="cuda")),
                dict(scales=torch.zeros(4, 2, device="cuda"))):
        with pytest.raises((ValueError, T.TTTError)):
            T.ttt_forward_rmsnorm_e4m3(**(dict(x=x, weight=w) | bad))
    with pytest.raises(T.TTTError):
        T.ttt_forward_rmsnorm_e4m3(x, w, group=16)
    d_y = torch.zeros_like(x)
    for bad in (dict(d_x=torch.zeros_like(x)), dict(p=0.5), dict(d_sum=res[:2]), dict(d_y=d_y[:2])):
        with pytest.raises((ValueError, TypeError)):
            T.ttt_backward_rmsnorm(**(dict(s=x, weight=w, d_y=d_y) | bad))
    for bad in (dict(d_s=d_y), dict(p=0.5, rng=rng, d_x=d_y), dict(eps=float("inf")), dict(d_weight=w)):
        with pytest.raises(T.TTTError):
            T.ttt_backward_rmsnorm(**(dict(s=x, weight=w, d_y=d_y) | bad))


def test_replayed_with_new_masks_and_on_another_stream():
    i = Inputs(21, "bf16")
    x, w, res, d_y = i.normal(130, 768), i.param(768), i.normal(130, 768), i.normal(130, 768)
    y, s, d_s, d_x = (torch.empty_like(x) for _ in range(4))
    d_w, rng = torch.empty_like(w), rng_of(77, 0)

    def call():
        T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=0.5, rng=rng, sum_out=s, y=y)
        T.ttt_backward_rmsnorm(s, w, d_y, EPS, p=0.5, rng=rng, d_s=d_s, d_x=d_x, d_weight=d_w)

    outs = [y, s, d_s, d_x, d_w]
    replays(call, outs, lambda: T.ttt_forward_rmsnorm(d_y, w))
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [*T.ttt_forward_rmsnorm(x, w, EPS, residual=res, p=0.5, rng=rng, stream=side)]
    got += T.ttt_backward_rmsnorm(got[1], w, d_y, EPS, p=0.5, rng=rng, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        rng[1] += T.dropout_counters(x)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert rng.tolist() == [77, (k + 1) * 130 * 96]
        assert torch.equal(s != res, (factors(77, k * 130 * 96, 0.5, 130, 768) > 0) & (s != res))
        assert float((s != res).double().mean()) > 0.45
