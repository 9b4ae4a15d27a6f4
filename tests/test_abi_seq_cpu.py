"""The C ABI of the block operators (include/ttt_seq.h) without a GPU: every declared symbol is exported and
bound, workspaces are sized, and bad arguments are refused before anything is launched.

Every call below that passes pointers is built to FAIL VALIDATION (the pointers are fake but never
dereferenced, because the library validates all arguments before it enqueues work).
"""
import os
import re

import pytest

import test_sequence_layers_amd as T
from test_sequence_layers_amd import ttt as binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = T.TTT_F32, T.TTT_BF16
BIG = 1 << 62
P = [(i + 1) << 40 for i in range(32)]  # far apart, aligned


def _declared():
    src = open(os.path.join(ROOT, "include", "ttt_seq.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(ttt_[a-z0-9_]+)\s*\(", src)))


def test_every_declared_symbol_is_exported_and_bound():
    names = _declared()
    assert len(names) == 12
    lib = T.load_library()
    for name in names:
        assert hasattr(lib, name), name
        assert name in binding.SIGNATURES, name
        if not name.endswith("_workspace"):
            assert callable(getattr(T, name)), name


def _norm(dt=BF16, M=8, H=2, D=64, eps=1e-5, x=P[0], xs=128, w=P[1], b=P[2], y=P[3]):
    return T.load_library().ttt_forward_layernorm(dt, M, H, D, eps, x, xs, w, b, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=7), INVALID), (dict(M=0), INVALID), (dict(H=-1), INVALID), (dict(D=0), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(xs=127), INVALID), (dict(xs=BIG), INVALID), (dict(x=P[0] + 1), INVALID), (dict(w=P[1] + 2), INVALID),
    (dict(y=P[0]), INVALID), (dict(y=P[2]), INVALID), (dict(D=16385, xs=40000), UNSUPPORTED),
    (dict(H=65536, xs=BIG), UNSUPPORTED), (dict(H=4096, D=4097, xs=BIG), UNSUPPORTED), (dict(M=1 << 30, H=2), UNSUPPORTED)])
def test_layernorm_refusals(kw, want):
    assert _norm(**kw) == want


def _norm_bwd(dt=BF16, M=8, H=2, D=64, eps=1e-5, x=P[0], xs=128, w=P[1], dy=P[2], dx=P[3], dw=P[4], db=P[5], ws=P[6],
              n=1 << 30):
    return T.load_library().ttt_backward_layernorm(dt, M, H, D, eps, x, xs, w, dy, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(dx=P[2]), INVALID),
    (dict(db=P[4]), INVALID), (dict(dw=P[0]), INVALID), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE),
    (dict(ws=P[6] + 4), INVALID), (dict(ws=P[0]), INVALID), (dict(ws=P[3]), INVALID), (dict(eps=float("inf")), INVALID)])
def test_layernorm_backward_refusals(kw, want):
    assert _norm_bwd(**kw) == want


def _conv(dt=BF16, B=2, N=10, C=64, K=4, silu=1, x=P[0], xs=64, w=P[1], b=P[2], state=P[3], lengths=P[4], y=P[5],
          so=P[6]):
    return T.load_library().ttt_forward_conv1d(dt, B, N, C, K, silu, x, xs, w, b, state, lengths, y, so, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=-1), INVALID), (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=1), UNSUPPORTED),
    (dict(K=5), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(N=(1 << 22) + 1), UNSUPPORTED), (dict(silu=2), INVALID),
    (dict(C=(1 << 20) + 1, xs=1 << 21), UNSUPPORTED), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(xs=63), INVALID), (dict(y=P[0]), INVALID), (dict(so=P[3]), INVALID),
    (dict(so=P[5] + 64), INVALID), (dict(lengths=P[4] + 2), INVALID), (dict(state=P[3] + 1), INVALID)])
def test_conv1d_refusals(kw, want):
    assert _conv(**kw) == want


def _conv_step(dt=BF16, B=2, C=64, K=4, silu=0, x=P[0], xs=64, w=P[1], b=P[2], state=P[3], y=P[4], so=P[5]):
    return T.load_library().ttt_step_conv1d(dt, B, C, K, silu, x, xs, w, b, state, y, so, None)


@pytest.mark.parametrize("kw,want", [
    (dict(state=None), INVALID), (dict(so=None), INVALID), (dict(so=P[3] + 2), INVALID), (dict(y=P[3]), INVALID),
    (dict(state=None, so=None), INVALID), (dict(K=5), UNSUPPORTED), (dict(silu=-1), INVALID)])
def test_conv1d_step_refusals(kw, want):
    assert _conv_step(**kw) == want


def _conv_bwd(dt=F32, B=2, N=10, C=64, K=4, silu=1, x=P[0], xs=64, w=P[1], b=P[2], state=P[3], lengths=P[4], dy=P[5],
              dx=P[6], dw=P[7], db=P[8], ds=P[9], ws=P[10], n=1 << 30):
    return T.load_library().ttt_backward_conv1d(dt, B, N, C, K, silu, x, xs, w, b, state, lengths, dy, dx, dw, db, ds, ws,
                                                n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(state=None), INVALID),
    (dict(dx=P[5]), INVALID), (dict(ds=P[3]), INVALID), (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE),
    (dict(ws=P[7]), INVALID), (dict(K=9), UNSUPPORTED)])
def test_conv1d_backward_refusals(kw, want):
    assert _conv_bwd(**kw) == want


def _scan(dt=BF16, B=2, N=10, C=64, S=16, G=1, sp=1, u=P[0], us=64, de=P[1], ds=64, A=P[2], bm=P[3], bs=16, cm=P[4],
          cs=16, D=P[5], db=P[6], z=P[7], zs=64, h0=P[8], lengths=P[9], y=P[10], ho=P[11], ws=P[12], n=1 << 30):
    return T.load_library().ttt_forward_selective_scan(dt, B, N, C, S, G, sp, u, us, de, ds, A, bm, bs, cm, cs, D, db, z,
                                                       zs, h0, lengths, y, ho, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), INVALID), (dict(B=-1), INVALID), (dict(C=0), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID),
    (dict(S=12), UNSUPPORTED), (dict(S=128, bs=128, cs=128), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(N=(1 << 22) + 1), UNSUPPORTED), (dict(B=60000, N=1 << 22), UNSUPPORTED), (dict(sp=2), INVALID),
    (dict(u=None), INVALID), (dict(de=None), INVALID), (dict(A=None), INVALID), (dict(bm=None), INVALID),
    (dict(cm=None), INVALID), (dict(y=None), INVALID), (dict(us=63), INVALID), (dict(bs=15), INVALID),
    (dict(bs=17), INVALID),            # bf16: an odd stride splits dwords
    (dict(cm=P[4] + 2), INVALID),      # bf16: not 4-byte aligned
    (dict(y=P[0]), INVALID), (dict(ho=P[8]), INVALID), (dict(y=P[7] + 128), INVALID), (dict(zs=1), INVALID),
    (dict(ws=None, N=100000), WORKSPACE), (dict(n=64, N=100000), WORKSPACE), (dict(ws=P[0], N=100000), INVALID)])
def test_scan_refusals(kw, want):
    assert _scan(**kw) == want


def _scan_step(dt=BF16, B=2, C=64, S=16, G=1, sp=1, u=P[0], us=64, de=P[1], ds=64, A=P[2], bm=P[3], bs=16, cm=P[4], cs=16,
               D=P[5], db=P[6], z=P[7], zs=64, h=P[8], y=P[9], ho=P[10]):
    return T.load_library().ttt_step_selective_scan(dt, B, C, S, G, sp, u, us, de, ds, A, bm, bs, cm, cs, D, db, z, zs, h, y,
                                                    ho, None)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), INVALID), (dict(ho=None), INVALID), (dict(ho=P[8] + 16), INVALID), (dict(y=P[8]), INVALID),
    (dict(h=None, ho=None), INVALID), (dict(S=4), UNSUPPORTED), (dict(bm=P[3] + 2), INVALID)])
def test_scan_step_refusals(kw, want):
    assert _scan_step(**kw) == want


def _scan_bwd(dt=BF16, B=2, N=10, C=64, S=16, G=1, sp=1, u=P[0], us=64, de=P[1], ds=64, A=P[2], bm=P[3], bs=16, cm=P[4],
              cs=16, D=P[5], db=P[6], z=P[7], zs=64, h0=P[8], lengths=P[9], dy=P[10], du=P[11], dd=P[12], dA=P[13], dB=P[14],
              dC=P[15], dD=P[16], ddb=P[17], dz=P[18], dh=P[19], ws=P[20], n=1 << 40):
    return T.load_library().ttt_backward_selective_scan(dt, B, N, C, S, G, sp, u, us, de, ds, A, bm, bs, cm, cs, D, db, z, zs,
                                                        h0, lengths, dy, du, dd, dA, dB, dC, dD, ddb, dz, dh, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(du=None), INVALID), (dict(dA=None), INVALID), (dict(dB=None), INVALID),
    (dict(dz=None), INVALID),          # z without d_z
    (dict(z=None), INVALID),           # d_z without z
    (dict(du=P[0]), INVALID), (dict(dB=P[14], dC=P[14]), INVALID), (dict(dh=P[8]), INVALID), (dict(ws=None), WORKSPACE),
    (dict(n=1024), WORKSPACE), (dict(ws=P[11]), INVALID), (dict(S=24), UNSUPPORTED), (dict(G=5), INVALID)])
def test_scan_backward_refusals(kw, want):
    assert _scan_bwd(**kw) == want


def test_workspace_sizes():
    lib = T.load_library()
    norm, conv = lib.ttt_backward_layernorm_workspace, lib.ttt_backward_conv1d_workspace
    fwd, bwd = lib.ttt_forward_selective_scan_workspace, lib.ttt_backward_selective_scan_workspace
    assert norm(BF16, 12544, 1, 384) > 0 and norm(BF16, 12544, 1, 384) % 256 == 0
    assert norm(BF16, 1 << 20, 1, 384) == norm(BF16, 1 << 21, 1, 384)  # the partial rows are capped
    assert norm(BF16, 0, 1, 384) == 0 and norm(BF16, 8, 1, 20000) == 0 and norm(9, 8, 1, 64) == 0
    assert conv(BF16, 2, 100, 64, 4) > 0 and conv(BF16, 2, 100, 64, 5) == 0
    assert fwd(BF16, 1, 24, 64, 16, 1) == 0                            # one segment
    assert fwd(BF16, 1, 65536, 64, 16, 1) > 0 and fwd(BF16, 1, 65536, 64, 12, 1) == 0
    assert fwd(BF16, 1, 65536, 64, 16, 3) == 0
    assert bwd(BF16, 1, 64, 64, 16, 1) > 0 and bwd(F32, 1, 64, 64, 16, 5) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 3, 8), torch.zeros(8, 4)
    with pytest.raises(TypeError):
        T.ttt_forward_layernorm(x, torch.zeros(8))
    with pytest.raises(TypeError):
        T.ttt_forward_conv1d(x, w)
    with pytest.raises(TypeError):
        T.ttt_step_conv1d(x[:, 0], w, state=torch.zeros(2, 3, 8))
    with pytest.raises(TypeError):
        T.ttt_forward_selective_scan(x, x, torch.zeros(8, 16), torch.zeros(2, 3, 1, 16), torch.zeros(2, 3, 1, 16))
