"""The C ABI of the residual block's operators (include/ttt_lm.h) without a GPU: every declared symbol is exported and bound,
workspaces are sized, and bad arguments are refused before anything is launched.

Every call below that passes pointers is built to FAIL VALIDATION (the pointers are fake but never dereferenced,
because the library validates all arguments before it enqueues work).
"""
import os
import re

import pytest

import test_sequence_layers_amd as T
from test_sequence_layers_amd import ttt as binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F32, BF16 = T.TTT_F32, T.TTT_BF16
BIG = 1 << 62
P = [(i + 1) << 40 for i in range(32)]  # far apart, aligned


def test_every_declared_symbol_is_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "ttt_lm.h")).read()
    names = sorted(set(re.findall(r"\b(ttt_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S))))
    assert len(names) == 12
    lib = T.load_library()
    for name in names:
        assert hasattr(lib, name), name
        assert name in binding.SIGNATURES, name
        if not name.endswith("_workspace") and name != "ttt_dropout_counters":
            assert callable(getattr(T, name)), name


def _norm(dt=BF16, M=8, H=1, D=64, eps=1e-5, x=P[0], xs=64, res=P[1], p=0.1, rng=P[2], w=P[3], s=P[4], y=P[5]):
    return T.load_library().ttt_forward_rmsnorm(dt, M, H, D, eps, x, xs, res, p, rng, w, s, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=7), INVALID), (dict(M=0), INVALID), (dict(H=-1), INVALID), (dict(D=0), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(xs=63), INVALID), (dict(xs=BIG), INVALID), (dict(x=P[0] + 1), INVALID), (dict(w=P[3] + 2), INVALID),
    (dict(y=P[0]), INVALID), (dict(y=P[1]), INVALID), (dict(s=P[0]), INVALID), (dict(s=P[1] + 16), INVALID), (dict(s=None), INVALID),
    (dict(res=None), INVALID), (dict(res=None, s=None), INVALID), (dict(rng=None), INVALID), (dict(rng=P[2] + 4), INVALID),
    (dict(y=P[2]), INVALID), (dict(p=1.0), INVALID), (dict(p=-1e-9), INVALID), (dict(p=float("nan")), INVALID),
    (dict(p=65535.6 / 65536), INVALID), (dict(D=16385, xs=40000), UNSUPPORTED), (dict(H=65536, xs=BIG), UNSUPPORTED),
    (dict(H=2, xs=128), UNSUPPORTED), (dict(M=1 << 30, H=2), UNSUPPORTED)])
def test_rmsnorm_refusals(kw, want):
    assert _norm(**kw) == want


def _e4m3(dt=BF16, M=8, H=1, D=256, group=128, eps=1e-5, x=P[0], xs=256, res=P[1], w=P[3], s=P[4], y=P[5], sc=P[6]):
    return T.load_library().ttt_forward_rmsnorm_e4m3(dt, M, H, D, group, eps, x, xs, res, w, s, y, sc, None)


@pytest.mark.parametrize("kw,want", [
    (dict(group=0), INVALID), (dict(group=96), INVALID), (dict(group=16), UNSUPPORTED), (dict(sc=None), INVALID), (dict(sc=P[5]), INVALID),
    (dict(sc=P[6] + 2), INVALID), (dict(x=P[0] + 1), INVALID), (dict(xs=255), INVALID), (dict(res=P[1] + 1), INVALID),
    (dict(w=P[3] + 2), INVALID), (dict(s=P[1] + 8), INVALID), (dict(y=P[4]), INVALID),
    (dict(s=None), INVALID), (dict(H=2, D=128), UNSUPPORTED)])
def test_rmsnorm_e4m3_refusals(kw, want):
    assert _e4m3(**kw) == want


def _norm_bwd(dt=BF16, M=8, H=1, D=64, eps=1e-5, s=P[0], ss=64, w=P[1], dy=P[2], dsum=P[3], p=0.1, rng=P[4], ds=P[5], dx=P[6],
              dw=P[7], ws=P[8], n=1 << 30):
    return T.load_library().ttt_backward_rmsnorm(dt, M, H, D, eps, s, ss, w, dy, dsum, p, rng, ds, dx, dw, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(ds=None), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(p=0.0), INVALID),
    (dict(rng=None), INVALID), (dict(ds=P[2]), INVALID), (dict(ds=P[3] + 16), INVALID), (dict(dx=P[3]), INVALID), (dict(dx=P[5]), INVALID),
    (dict(dw=P[0]), INVALID), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=P[8] + 4), INVALID), (dict(ws=P[0]), INVALID),
    (dict(ws=P[6]), INVALID), (dict(H=2, ss=128), UNSUPPORTED), (dict(eps=float("inf")), INVALID)])
def test_rmsnorm_backward_refusals(kw, want):
    assert _norm_bwd(**kw) == want


def _drop(dt=BF16, M=8, C=64, p=0.1, rng=P[0], x=P[1], xs=64, res=P[2], y=P[3]):
    return T.load_library().ttt_forward_dropout(dt, M, C, p, rng, x, xs, res, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), INVALID), (dict(M=0), INVALID), (dict(C=-1), INVALID), (dict(C=(1 << 24) + 1, xs=1 << 25), UNSUPPORTED),
    (dict(M=1 << 30, C=1 << 20, xs=1 << 20), UNSUPPORTED), (dict(p=1.0), INVALID), (dict(rng=None), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(x=None, y=None), INVALID), (dict(xs=63), INVALID), (dict(y=P[1] + 2), INVALID),
    (dict(y=P[1], xs=65), INVALID), (dict(y=P[2] + 2), INVALID), (dict(y=P[3] + 1), INVALID), (dict(y=P[0]), INVALID)])
def test_dropout_refusals(kw, want):
    assert _drop(**kw) == want


def test_dropout_backward_refusals():
    call = lambda p=0.1, rng=P[0], dy=P[1], dx=P[2]: T.load_library().ttt_backward_dropout(F32, 4, 8, p, rng, dy, dx, None)  # noqa: E731
    assert call(dy=None) == INVALID and call(dx=None) == INVALID and call(dx=P[1] + 4) == INVALID and call(rng=None) == INVALID


def test_dropout_counters():
    count = T.load_library().ttt_dropout_counters
    assert [count(3, c) for c in (1, 8, 9, 768)] == [3, 3, 6, 288] and count(0, 8) == 0
    assert count((1 << 31) - 1, 1 << 24) == ((1 << 31) - 1) << 21


def _rec(dt=BF16, B=2, N=1000, C=64, scale=8.0, x=P[0], xs=64, r=P[1], rs=64, i=P[2], i_s=64, lam=P[3], h0=P[4], lengths=P[5], y=P[6],
         st=P[7], ho=P[8], ws=P[9], n=1 << 40):
    return T.load_library().ttt_forward_gated_recurrence(dt, B, N, C, scale, x, xs, r, rs, i, i_s, lam, h0, lengths, y, st, ho, ws,
                                                         n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), INVALID), (dict(B=-1), INVALID), (dict(N=0), INVALID), (dict(C=0), INVALID), (dict(B=65536), UNSUPPORTED),
    (dict(N=(1 << 22) + 1), UNSUPPORTED), (dict(C=(1 << 20) + 1, xs=1 << 21, rs=1 << 21, i_s=1 << 21), UNSUPPORTED),
    (dict(B=60000, N=1 << 22), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(x=None), INVALID), (dict(r=None), INVALID), (dict(i=None), INVALID), (dict(lam=None), INVALID), (dict(y=None), INVALID),
    (dict(xs=63), INVALID), (dict(rs=1), INVALID), (dict(i_s=BIG), INVALID), (dict(x=P[0] + 1), INVALID), (dict(lam=P[3] + 2), INVALID),
    (dict(y=P[0]), INVALID), (dict(ho=P[4]), INVALID), (dict(st=P[8]), INVALID), (dict(st=P[6] + 256), INVALID)])
def test_recurrence_refusals(kw, want):
    assert _rec(**kw) == want


def _rec_step(dt=BF16, B=2, C=64, scale=8.0, x=P[0], xs=64, r=P[1], rs=64, i=P[2], i_s=64, lam=P[3], h=P[4], y=P[5], ho=P[6]):
    return T.load_library().ttt_step_gated_recurrence(dt, B, C, scale, x, xs, r, rs, i, i_s, lam, h, y, ho, None)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), INVALID), (dict(ho=None), INVALID), (dict(h=None, ho=None), INVALID), (dict(ho=P[4] + 16), INVALID),
    (dict(y=P[4]), INVALID), (dict(y=P[0]), INVALID), (dict(B=65536), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(lam=None), INVALID)])
def test_recurrence_step_refusals(kw, want):
    assert _rec_step(**kw) == want


def _rec_bwd(dt=BF16, B=2, N=1000, C=64, scale=8.0, x=P[0], xs=64, r=P[1], rs=64, i=P[2], i_s=64, lam=P[3], h0=P[4], lengths=P[5],
             st=P[6], dy=P[7], dx=P[8], dr=P[9], di=P[10], dl=P[11], dh=P[12], ws=P[13], n=1 << 40):
    return T.load_library().ttt_backward_gated_recurrence(dt, B, N, C, scale, x, xs, r, rs, i, i_s, lam, h0, lengths, st, dy, dx, dr,
                                                          di, dl, dh, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dr=None), INVALID), (dict(di=None), INVALID), (dict(dl=None), INVALID),
    (dict(dx=P[7]), INVALID), (dict(dr=P[8]), INVALID), (dict(dh=P[4]), INVALID), (dict(st=P[8]), INVALID), (dict(st=P[6] + 2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(n=64), WORKSPACE), (dict(ws=P[8]), INVALID), (dict(ws=P[13] + 8), INVALID),
    (dict(scale=0.0), INVALID), (dict(B=65536), UNSUPPORTED)])
def test_recurrence_backward_refusals(kw, want):
    assert _rec_bwd(**kw) == want


def test_workspace_sizes():
    lib = T.load_library()
    norm, fwd, bwd = (lib.ttt_backward_rmsnorm_workspace, lib.ttt_forward_gated_recurrence_workspace,
                      lib.ttt_backward_gated_recurrence_workspace)
    assert norm(BF16, 12544, 1, 384) > 0 and norm(BF16, 12544, 1, 384) % 256 == 0
    assert norm(BF16, 0, 1, 384) == 0 and norm(BF16, 8, 1, 20000) == 0 and norm(9, 8, 1, 64) == 0
    assert fwd(BF16, 0, 10, 64) == 0 and fwd(BF16, 1, (1 << 22) + 1, 64) == 0
    for kept in (0, 1):
        assert bwd(BF16, 4, 8192, 768, kept) > 0 and bwd(BF16, 4, 8192, 768, kept) % 256 == 0 and bwd(BF16, 4, 8192, 0, kept) == 0


def _channels_a_lane(B, N, C, dt):
    """Of the forward recurrence, from its workspace: 16 words for each column of 64 or 128 channels of a sequence, one for each channel
    of its tiles (of 128 tokens in bf16, 64 in fp32) and groups of 16 tiles, 8 bytes each."""
    need = T.load_library().ttt_forward_gated_recurrence_workspace(dt, B, N, C)
    tiles = -(-N // (128 if dt == BF16 else 64))
    fits = [V for V in (1, 2) if (8 * B * -(-C // (64 * V)) * (16 + 64 * V * (tiles + -(-tiles // 16))) + 255) // 256 * 256 == need]
    assert len(fits) == 1, (B, N, C, need)
    return fits[0]


@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_channel_of_the_recurrence_has_one_workgroup(dt):
    """With two channels a lane the last of an odd width is computed with the one before it, which has to be of the same column: a
    column forms its decays by all its channels, so two of them need not give the same bits for it."""
    seen = set()
    for C in [*range(1, 400), 511, 512, 513, 514, 769, 1023, 1024, 1025, 2049, 65537]:
        V = _channels_a_lane(300, 9000, C, dt) if C < 5000 else _channels_a_lane(2, 9000, C, dt)
        seen.add(V)
        assert V == 1 or C % 128 != 1, C
    assert seen == {1, 2}


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w, rng = torch.zeros(2, 3, 8), torch.zeros(8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: T.ttt_forward_rmsnorm(x, w), lambda: T.ttt_forward_rmsnorm_e4m3(x, w), lambda: T.ttt_backward_rmsnorm(x, w, x),
                 lambda: T.ttt_forward_dropout(x, 0.5, rng), lambda: T.ttt_backward_dropout(x, 0.5, rng),
                 lambda: T.ttt_forward_gated_recurrence(x, x, x, w), lambda: T.ttt_step_gated_recurrence(x[0], x[0], x[0], w, h=x[0]),
                 lambda: T.ttt_backward_gated_recurrence(x, x, x, w, x)):
        with pytest.raises(TypeError):
            call()
    assert T.dropout_counters(x) == 6
