"""Host-side checks of the long-context operators (no GPU): every refusal comes back as a
status or an exception before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: checks fail first
ODD = ctypes.c_void_p(0x100004)
BIG = ctypes.c_void_p(0x40000000)


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_96_gb300 import build
    build.build()
    from paged_kv_cache_96_gb300 import binding
    return binding


def _summarize(B, **kw):
    a = dict(codes=FAKE, scales=FAKE, kc=FAKE, bt=FAKE, mb=4, ctx=FAKE, qs=FAKE, S=2, N=8, bs=16,
             K=2, D=128, dt=1)
    a.update(kw)
    return B.lib().pa_summarize_blocks(*a.values(), None, None)


def _select(B, **kw):
    a = dict(sel=FAKE, k=8, q=FAKE, codes=FAKE, scales=FAKE, bt=FAKE, mb=64, seq=FAKE, pos=FAKE,
             maxctx=1024, first=1, last=1, T=2, S=2, H=8, K=2, D=128, bs=16, N=80, dt=1)
    a.update(kw)
    return B.lib().pa_select_blocks(*a.values(), None, None)


def _sparse(B, fp8=False, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=8, seq=FAKE, pos=FAKE, sel=FAKE, k=8,
             T=3, S=2, H=8, K=2, D=128, bs=16, N=8, scale=0.1)
    tail = dict(P=0, ws=None, wsb=0, dt=1)
    scales = [kw.pop("k_scale", 1.0), kw.pop("v_scale", 1.0)] if fp8 else []
    for k, v in kw.items():
        (tail if k in tail else a)[k] = v
    fn = B.lib().pa_decode_attention_sparse_fp8 if fp8 else B.lib().pa_decode_attention_sparse
    return fn(*a.values(), *scales, *tail.values(), None, None)


def _weights(B, fp8=False, **kw):
    a = dict(out=FAKE, wo=FAKE, q=FAKE, kc=FAKE, vc=FAKE, w=FAKE, bt=FAKE, mb=8, ctx=FAKE,
             old=FAKE, maxctx=128, S=2, H=8, K=2, D=128, bs=16, N=8, scale=0.1)
    tail = dict(P=0, ws=BIG, wsb=1 << 30, dt=1)
    scales = [kw.pop("k_scale", 1.0), kw.pop("v_scale", 1.0)] if fp8 else []
    for k, v in kw.items():
        (tail if k in tail else a)[k] = v
    fn = B.lib().pa_decode_attention_weights_fp8 if fp8 else B.lib().pa_decode_attention_weights
    return fn(*a.values(), *scales, *tail.values(), None, None)


def _plan(B, **kw):
    a = dict(moves=FAKE, M=50, co=FAKE, no=FAKE, wo=FAKE, bt=FAKE, mb=8, ctx=FAKE, w=FAKE,
             free=FAKE, cnt=FAKE, maxctx=128, limit=100, budget=50, sinks=4, recent=10, S=2, bs=16,
             N=8)
    a.update(kw)
    return B.lib().pa_plan_eviction(*a.values(), None, None)


def _move(B, **kw):
    a = dict(kc=FAKE, vc=FAKE, moves=FAKE, n=5, N=8, bs=16, K=2, D=64, dt=1)
    a.update(kw)
    return B.lib().pa_move_tokens(*a.values(), None, None)


def refuses(call, status, *cases, **common):
    for kw in cases:
        assert call(**dict(common, **kw)) == status, kw


def test_summarize_refuses(B):
    f = lambda **kw: _summarize(B, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(S=-1), dict(N=0), dict(bs=0), dict(mb=0), dict(K=0),
            dict(D=0), dict(dt=3), dict(dt=-1), dict(codes=None), dict(scales=None),
            dict(kc=None), dict(bt=None), dict(ctx=None), dict(codes=ODD), dict(kc=ODD))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(D=96), dict(D=256), dict(bs=8), dict(bs=48),
            dict(bs=512), dict(N=1 << 28), dict(S=1 << 20, mb=1 << 12))
    assert f(S=0) == B.PA_OK


def test_select_refuses(B):
    f = lambda **kw: _select(B, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(k=0), dict(k=-1), dict(first=-1), dict(last=-1),
            dict(first=9), dict(first=5, last=4), dict(T=-1), dict(S=-1), dict(H=0), dict(K=0),
            dict(D=0), dict(bs=0), dict(N=0), dict(mb=0), dict(maxctx=-1), dict(H=6, K=4),
            dict(dt=2), dict(sel=None), dict(q=None), dict(codes=None), dict(scales=None),
            dict(bt=None), dict(seq=None), dict(pos=None), dict(q=ODD), dict(codes=ODD),
            dict(first=(1 << 31) - 1, last=(1 << 31) - 1))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(D=96), dict(bs=8), dict(bs=24), dict(bs=512),
            dict(H=34, K=2), dict(N=1 << 28), dict(mb=1 << 28))
    assert f(T=0) == B.PA_OK


@pytest.mark.parametrize("call", [_sparse, _weights])
@pytest.mark.parametrize("fp8", [False, True])
def test_attention_refuses(B, call, fp8):
    f = lambda **kw: call(B, fp8, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(S=-1), dict(H=0), dict(K=0), dict(D=0), dict(bs=0),
            dict(N=0), dict(mb=0), dict(H=6, K=4), dict(scale=float("nan")), dict(scale=3e38),
            dict(out=None), dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None),
            dict(out=ODD), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(dt=2), dict(dt=9),
            dict(P=-16))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(D=96), dict(bs=8), dict(bs=48), dict(bs=512),
            dict(H=34, K=2), dict(N=1 << 28), dict(mb=1 << 28), dict(mb=1 << 27), dict(P=24))
    if fp8:
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            refuses(f, B.PA_ERR_INVALID_ARG, dict(k_scale=bad), dict(v_scale=bad))
        refuses(f, B.PA_ERR_INVALID_ARG, dict(scale=1e30, k_scale=1e9))


def test_sparse_refuses(B):
    f = lambda **kw: _sparse(B, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(k=0), dict(T=-1), dict(seq=None), dict(pos=None),
            dict(sel=None))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(k=1 << 28), dict(T=1 << 30),
            dict(k=1 << 20, T=1 << 10, P=16, ws=BIG, wsb=1 << 62))
    assert f(T=0) == B.PA_OK and f(T=0, S=0) == B.PA_OK
    need = B.pa_sparse_workspace_bytes(3, 8, 2, 128, 8, 16, 16)
    assert need == B.pa_decode_workspace_bytes(3, 8, 2, 128, 128, 16) + 256
    assert B.pa_sparse_workspace_bytes(3, 8, 2, 128, 8, 16, 0) == 0
    assert B.pa_sparse_workspace_bytes(3, 8, 2, 128, 8, 16, 96) == 0       # a short rest joins
    assert B.pa_sparse_workspace_bytes(3, 8, 2, 128, 8, 16, 64) == \
        B.pa_decode_workspace_bytes(3, 8, 2, 128, 128, 64) + 256           # and partials
    refuses(f, B.PA_ERR_WORKSPACE, dict(), dict(ws=BIG, wsb=need - 1),
            dict(ws=ctypes.c_void_p(0x40000010), wsb=need), P=16)
    for bad in ((-1, 8, 2, 128, 8, 16, 16), (3, 8, 2, 128, 0, 16, 16), (3, 8, 2, 128, 8, 16, -1),
                (3, 8, 2, 128, 1 << 30, 16, 16)):
        assert B.pa_sparse_workspace_bytes(*bad) == 0


def test_weights_refuses(B):
    f = lambda **kw: _weights(B, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(maxctx=-1), dict(wo=None), dict(w=None), dict(ctx=None),
            dict(old=None))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(H=8192, K=512), dict(maxctx=(1 << 31) - 1))
    assert f(S=0) == B.PA_OK
    need = B.pa_weights_workspace_bytes(2, 8, 2, 128, 128, 0)
    counters = 1 << 20                                      # kept for calls with partitions
    assert need == counters + 3 * 256 + 2 * 8 * 128 * 4     # sums, partials, scores
    refuses(f, B.PA_ERR_WORKSPACE, dict(ws=None), dict(wsb=need - 1),
            dict(ws=ctypes.c_void_p(0x40000010)))
    need = B.pa_weights_workspace_bytes(2, 8, 2, 128, 128, 16)
    assert need == B.pa_decode_workspace_bytes(2, 8, 2, 128, 128, 16) + 256 + 2 * 8 * 128 * 4
    refuses(f, B.PA_ERR_WORKSPACE, dict(ws=None), dict(wsb=need - 1), P=16)
    for P in (0, 16):                                       # contexts of no token have counts
        need = B.pa_weights_workspace_bytes(2, 8, 2, 128, 0, P)
        assert need == counters + 3 * 256 + 2 * 8 * 16 * 4
        refuses(f, B.PA_ERR_WORKSPACE, dict(ws=None), dict(wsb=need - 1), dict(wsb=0), P=P, maxctx=0)
    for bad in ((-1, 8, 2, 128, 128, 16), (2, 8, 2, 128, -1, 16), (2, 8, 2, 128, 128, -16)):
        assert B.pa_weights_workspace_bytes(*bad) == 0


def test_plan_refuses(B):
    f = lambda **kw: _plan(B, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(S=-1), dict(M=-1), dict(M=49), dict(mb=0), dict(bs=0),
            dict(N=0), dict(maxctx=-1), dict(budget=0), dict(limit=49), dict(sinks=-1),
            dict(recent=-1), dict(sinks=51), dict(sinks=40, recent=11),
            dict(sinks=1, recent=(1 << 31) - 1), dict(moves=None), dict(co=None), dict(no=None),
            dict(wo=None), dict(bt=None), dict(ctx=None), dict(w=None), dict(free=None),
            dict(cnt=None))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(bs=24), dict(N=1 << 28), dict(mb=1 << 28),
            dict(M=(1 << 29) + 1))


def test_move_refuses(B):
    f = lambda **kw: _move(B, **kw)  # noqa: E731
    refuses(f, B.PA_ERR_INVALID_ARG, dict(n=-1), dict(N=0), dict(bs=0), dict(K=0), dict(D=0),
            dict(dt=3), dict(kc=None), dict(vc=None), dict(moves=None), dict(kc=ODD),
            dict(vc=ODD), dict(moves=ODD))
    refuses(f, B.PA_ERR_UNSUPPORTED, dict(K=1, D=4), dict(K=1, D=24, dt=2), dict(N=1 << 28),
            dict(n=(1 << 40) + 1), dict(K=1 << 14, D=1 << 10))
    assert f(n=0) == B.PA_OK


def z(*s, dt=torch.int32):
    return torch.zeros(s, dtype=dt)


def calls(B):
    """One call of each on host tensors of fitting shapes: (function, arguments)."""
    q, pool, w = z(4, 8, 64, dt=torch.bfloat16), z(8, 16, 2, 64, dt=torch.bfloat16), \
        z(8, 16, dt=torch.float32)
    codes, scales = z(8, 2, 2, 64, dt=torch.int8), z(8, 2, dt=torch.float32)
    return {
        "summarize": (B.pa_summarize_blocks, [codes, scales, pool, z(4, 2), z(4), z(5)]),
        "select": (B.pa_select_blocks, [z(4, 2, 3), q, codes, scales, z(4, 2), z(4), z(4), 32, 16]),
        "sparse": (B.pa_decode_attention_sparse, [q, q, pool, pool, z(4, 2), z(4), z(4),
                                                  z(4, 2, 3), 0.1]),
        "weights": (B.pa_decode_attention_weights, [q, w, q, pool, pool, w, z(4, 2), z(4), z(4),
                                                    32, 0.1, z(9)]),
        "plan": (B.pa_plan_eviction, [z(4, 9, 2), z(4), z(1), w, z(4, 2), z(4), w, z(8), z(1), 32,
                                      16, 8]),
        "move": (B.pa_move_tokens, [pool, pool, z(4, 9, 2)]),
    }


@pytest.mark.parametrize("name", ["summarize", "select", "sparse", "weights", "plan", "move"])
def test_binding_refuses_host_tensors_and_what_is_none(B, name):
    fn, args = calls(B)[name]
    with pytest.raises(ValueError, match="CUDA tensor"):
        fn(*args)
    for k, a in enumerate(args):
        if name == "summarize" and k == 5 or name == "weights" and k == 11:
            continue                                        # may be None
        bad = [None, "16", 1.5 if isinstance(a, int) else None] if not isinstance(a, float) \
            else [None, "x"]
        for x in bad:                                       # (the device may be looked at first)
            with pytest.raises((TypeError, ValueError)):
                fn(*[x if i == k else b for i, b in enumerate(args)])


@pytest.mark.parametrize("name,at,shape", [
    ("summarize", 0, (8, 2, 3, 64)), ("summarize", 0, (7, 2, 2, 64)), ("summarize", 1, (8, 3)),
    ("summarize", 2, (8, 16, 2)), ("summarize", 3, (3, 2)), ("summarize", 5, (4,)),
    ("select", 0, (4, 3, 3)), ("select", 0, (4, 2)), ("select", 1, (3, 8, 64)),
    ("select", 5, (5,)), ("select", 6, (3,)), ("select", 2, (8, 2, 2, 32)),
    ("sparse", 0, (4, 8, 32)), ("sparse", 5, (3,)), ("sparse", 6, (4, 1)), ("sparse", 7, (4, 8, 3)),
    ("sparse", 7, (3, 2, 3)), ("sparse", 3, (8, 16, 2, 32)),
    ("weights", 1, (8, 8)), ("weights", 5, (8,)), ("weights", 6, (3, 2)), ("weights", 8, (5,)),
    ("plan", 0, (4, 9)), ("plan", 0, (3, 9, 2)), ("plan", 0, (4, 9, 3)), ("plan", 1, (3,)),
    ("plan", 3, (8, 8)), ("plan", 5, (5,)), ("plan", 7, (7,)), ("plan", 8, (0,)),
    ("move", 1, (8, 16, 2, 32)), ("move", 2, (4, 9, 3)), ("move", 0, (8, 16, 2))])
def test_binding_refuses_shapes(B, name, at, shape):
    fn, args = calls(B)[name]
    args[at] = torch.zeros(shape, dtype=args[at].dtype)
    with pytest.raises(ValueError):
        fn(*args)


def test_binding_takes_integers_only(B):
    for f, good in ((B.pa_sparse_workspace_bytes, (3, 8, 2, 128, 8, 16, 16)),
                    (B.pa_weights_workspace_bytes, (2, 8, 2, 128, 128, 16))):
        assert f(*good) > 0
        for bad in (16.0, "16", None, np.float32(16)):
            for i in range(len(good)):
                with pytest.raises((TypeError, ctypes.ArgumentError)):
                    f(*[bad if i == k else x for k, x in enumerate(good)])
