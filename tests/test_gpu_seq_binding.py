"""The block operators' binding: what it takes, what it returns and what it keeps, on any thread, stream or mode."""
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

import test_sequence_layers_amd as T  # noqa: E402

pytestmark = pytest.mark.gpu


def _scan(B=2, N=70, C=65, S=16, G=1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return dict(u=r(B, N, C), delta=r(B, N, C), A=-r(C, S).abs() - 0.1, Bm=r(B, N, G, S), Cm=r(B, N, G, S), D=r(C),
                delta_bias=r(C), z=r(B, N, C))


def test_outputs_are_the_callers_or_new_ones():
    s = _scan()
    for out in (None, torch.empty_like(s["u"])):
        y = T.ttt_forward_selective_scan(**s, y=out)
        assert y is out if out is not None else (y.is_contiguous() and not y.requires_grad)
    x, w, b = s["u"], torch.ones(65, device="cuda"), torch.zeros(65, device="cuda")
    dx, dw, db = (torch.empty_like(t) for t in (x, w, b))
    got = T.ttt_backward_layernorm(x, w, s["z"], d_x=dx, d_weight=dw, d_bias=db)
    assert type(got) is tuple and got[0] is dx and got[1] is dw and got[2] is db
    for a, c in zip(got, T.ttt_backward_layernorm(x, w, s["z"])):
        assert torch.equal(a, c)
    cw = torch.ones(65, 3, device="cuda")
    assert T.ttt_backward_conv1d(x, cw, None, s["z"])[2:] == (None, None)
    assert T.ttt_backward_selective_scan(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["z"])[5:] == (None,) * 4


def test_nothing_is_kept():
    """Neither references to the tensors nor device memory."""
    s = _scan()
    x, w, y = s["u"], torch.ones(65, device="cuda"), torch.empty_like(s["u"])
    torch.cuda.synchronize()

    def calls():
        T.ttt_forward_layernorm(x, w, y=y)
        T.ttt_backward_layernorm(x, w, y)
        T.ttt_forward_selective_scan(**s)
        T.ttt_backward_selective_scan(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], y, z=s["z"])
        for bad in (dict(weight=w[:4]), dict(y=s["A"]), dict(bias=0)):
            with pytest.raises((ValueError, TypeError)):
                T.ttt_forward_layernorm(**(dict(x=x, weight=w) | bad))

    calls()
    counts = [sys.getrefcount(t) for t in (x, w, y, *s.values())]
    held = torch.cuda.memory_allocated()
    for _ in range(20):
        calls()
    assert [sys.getrefcount(t) for t in (x, w, y, *s.values())] == counts
    assert torch.cuda.memory_allocated() == held
    none = sys.getrefcount(None)
    for _ in range(2000):
        T.ttt_backward_conv1d(x, torch.ones(65, 3, device="cuda"), None, y)
    assert abs(sys.getrefcount(None) - none) < 500  # (its count moves by a few in either direction)


def test_parameters_and_inference_mode():
    x = torch.randn(3, 5, 64, device="cuda")
    w = torch.nn.Parameter(torch.randn(64, device="cuda"))
    want = T.ttt_forward_layernorm(x, w.detach())
    got = T.ttt_forward_layernorm(x.requires_grad_(), w)
    assert torch.equal(got, want) and not got.requires_grad and got.grad_fn is None
    dw = T.ttt_backward_layernorm(x, w, want)[1]
    assert type(dw) is torch.Tensor and not dw.requires_grad
    with torch.inference_mode():
        assert torch.equal(T.ttt_forward_layernorm(x, w), want)


def test_negated_views_are_refused():
    x, w = torch.ones(3, 64, device="cuda"), torch.ones(64, device="cuda")
    neg = torch._neg_view(x)
    for bad in (dict(x=neg), dict(y=neg)):
        with pytest.raises(ValueError):
            T.ttt_forward_layernorm(**(dict(x=x, weight=w) | bad))


def test_a_call_runs_on_the_current_or_the_given_stream():
    """In order behind what its stream holds: the inputs are written there, and read after."""
    s, side = _scan(4, 3000, 256), torch.cuda.Stream()
    want = T.ttt_forward_selective_scan(**s)
    torch.cuda.synchronize()
    for given in (False, True):
        late = {k: torch.zeros_like(v) for k, v in s.items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                burn = torch.ones(1 << 24, device="cuda").sqrt_()
            for k, v in s.items():
                late[k].copy_(v)
            if not given:
                got = T.ttt_forward_selective_scan(**late)
        if given:
            got = T.ttt_forward_selective_scan(**late, stream=side)
        assert torch.cuda.current_stream() != side
        side.synchronize()
        assert torch.equal(got, want), given
        del burn


def test_calls_from_several_threads():
    """Each on a stream of its own, at once: the results of a call alone."""
    cases = [_scan(seed=i, N=100 + 50 * i) for i in range(4)]
    want = [T.ttt_forward_selective_scan(**s) for s in cases]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(cases))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(50):
                y = T.ttt_forward_selective_scan(**cases[i], stream=stream)
            stream.synchronize()
            if not torch.equal(y, want[i]):
                bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("B,N,C,S,G,dtype", [(1, 700, 130, 8, 2, "bf16"), (2, 1000, 64, 16, 1, "fp32"), (3, 257, 100, 32, 1, "bf16"),
                                             (1, 5000, 64, 64, 1, "fp32"), (2, 49, 65, 64, 1, "bf16")])
def test_workspaces_are_enough_and_not_left(B, N, C, S, G, dtype):
    """Each call with a workspace of exactly the size that is asked for, inside a larger buffer: the same results as with
    a workspace of the binding's own, and the bytes around it as they were. With lengths as without."""
    print(f"workspaces B={B} N={N} C={C} S={S} G={G} {dtype}", flush=True)
    io, code, lib = (torch.bfloat16, T.TTT_BF16, T.load_library()) if dtype == "bf16" else (torch.float32, T.TTT_F32, T.load_library())
    s = {k: v if k in ("A", "D", "delta_bias") else v.to(io) for k, v in _scan(B, N, C, S, G).items()}
    lengths = torch.tensor([N - 3 * b for b in range(B)], dtype=torch.int32, device="cuda")
    u, w, cw, dy = s["u"], torch.ones(C, device="cuda"), torch.ones(C, 4, device="cuda"), s["z"]
    for need, call in (
            (lib.ttt_forward_selective_scan_workspace(code, B, N, C, S, G), lambda **k: (T.ttt_forward_selective_scan(**s, **k),)),
            (lib.ttt_forward_selective_scan_workspace(code, B, N, C, S, G),
             lambda **k: (T.ttt_forward_selective_scan(**s, lengths=lengths, **k),)),
            (lib.ttt_backward_selective_scan_workspace(code, B, N, C, S, G),
             lambda **k: T.ttt_backward_selective_scan(**s, d_y=dy, lengths=lengths, **k)),
            (lib.ttt_backward_conv1d_workspace(code, B, N, C, 4), lambda **k: T.ttt_backward_conv1d(u, cw, w, dy, silu=True, **k)),
            (lib.ttt_backward_layernorm_workspace(code, B * N, 1, C), lambda **k: T.ttt_backward_layernorm(u, w, dy, **k))):
        around = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        got, want = call(workspace=around[4096:4096 + need] if need else None), call()
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))
        assert bool((around[:4096] == 0x5A).all()) and bool((around[4096 + need:] == 0x5A).all())
        if need:
            with pytest.raises(T.TTTError):
                call(workspace=around[4096:4096 + need - 256])
