"""Host-side checks of the serving-step operators through the C ABI (no GPU):
every refusal comes back as a status before anything is launched."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: checks fail first
FAKE2 = ctypes.c_void_p(0x900000)
ODD = ctypes.c_void_p(0x100002)
AXES = (ctypes.c_int32 * 64)(*([0] * 40 + [1] * 12 + [2] * 12))


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_96_gb300 import build
    build.build()
    from paged_kv_cache_96_gb300 import binding
    return binding


def _maps(B, **kw):
    a = dict(qs=FAKE, seq=FAKE, pos=FAKE, slot=FAKE, cout=FAKE, fout=FAKE, bt=FAKE, mb=4,
             ctx=FAKE, ql=FAKE2, free=FAKE, cnt=FAKE, S=2, T=8, bs=16, N=8)
    a.update(kw)
    return B.lib().pa_build_step_maps(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(S=-1), dict(T=-1), dict(mb=0), dict(bs=0), dict(N=0), dict(qs=None), dict(free=None),
    dict(cnt=None), dict(fout=None), dict(seq=None), dict(pos=None), dict(slot=None),
    dict(cout=None), dict(bt=None), dict(ctx=None), dict(ql=None), dict(ql=FAKE)],
    ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_step_maps_refuses(B, kw):
    assert _maps(B, **kw) == B.PA_ERR_INVALID_ARG


def test_step_maps_limits(B):
    assert _maps(B, bs=1 << 20, N=1 << 12) == B.PA_ERR_UNSUPPORTED
    assert _maps(B, bs=1 << 20, mb=1 << 12) == B.PA_ERR_UNSUPPORTED
    assert _maps(B, T=(1 << 30) + 1) == B.PA_ERR_UNSUPPORTED


def _rope(B, fp8=False, **kw):
    a = dict(qo=FAKE2, qos=1024, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, kc=FAKE,
             vc=FAKE, slot=FAKE, pos=FAKE, axes=3, axis=AXES, freq=FAKE, rot=128, inter=0, T=4,
             H=8, K=2, D=128, bs=16, N=8, dt=1)
    scales = [kw.pop("k_scale", 1.0), kw.pop("v_scale", 1.0)] if fp8 else []
    a.update(kw)
    fn = B.lib().pa_rope_and_cache_fp8 if fp8 else B.lib().pa_rope_and_cache
    return fn(*a.values(), *scales, None, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(K=0), dict(D=0), dict(bs=0), dict(N=0), dict(axes=0),
    dict(rot=0), dict(rot=144), dict(inter=2), dict(dt=2), dict(dt=7), dict(qo=None),
    dict(q=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(slot=None),
    dict(pos=None), dict(freq=None), dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(v=ODD),
    dict(kc=ODD), dict(vc=ODD), dict(qs=1020), dict(qs=512), dict(ks=128), dict(qos=-1024),
    dict(vs=1 << 30), dict(axes=2),                       # a pair's axis past the axes
    dict(qo=ctypes.c_void_p(0x100010)),                   # output overlaps the query
    dict(qo=FAKE, qos=2048),                              # in place with another stride
    dict(qo=FAKE2, k=FAKE2)],                             # output overlaps the keys
    ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_rope_refuses(B, kw):
    assert _rope(B, **kw) == B.PA_ERR_INVALID_ARG
    assert _rope(B, fp8=True, **kw) == B.PA_ERR_INVALID_ARG


def test_rope_limits(B):
    for fp8 in (False, True):
        assert _rope(B, fp8, D=136) == B.PA_ERR_UNSUPPORTED
        assert _rope(B, fp8, D=272) == B.PA_ERR_UNSUPPORTED
        assert _rope(B, fp8, rot=24) == B.PA_ERR_UNSUPPORTED
        assert _rope(B, fp8, axes=256) == B.PA_ERR_UNSUPPORTED
        assert _rope(B, fp8, N=1 << 28) == B.PA_ERR_UNSUPPORTED
        assert _rope(B, fp8, T=0) == B.PA_OK
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert _rope(B, True, k_scale=bad) == B.PA_ERR_INVALID_ARG
        assert _rope(B, True, v_scale=bad) == B.PA_ERR_INVALID_ARG


def _decode(B, fp8=False, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=8, ctx=FAKE, maxctx=128, W=64, N=4,
             S=2, H=8, K=2, D=128, bs=16, NB=8, scale=0.1)
    tail = dict(P=0, ws=None, wsb=0, dt=1)
    scales = [kw.pop("k_scale", 1.0), kw.pop("v_scale", 1.0)] if fp8 else []
    for k, v in kw.items():
        (tail if k in tail else a)[k] = v
    fn = B.lib().pa_decode_attention_window_fp8 if fp8 else B.lib().pa_decode_attention_window
    return fn(*a.values(), *scales, *tail.values(), None, None)


def _chunk(B, fp8=False, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=8, qs=FAKE, ctx=FAKE, maxctx=128,
             W=64, N=4, S=2, T=9, H=8, K=2, D=128, bs=16, NB=8, scale=0.1)
    dt = kw.pop("dt", 1)
    scales = [kw.pop("k_scale", 1.0), kw.pop("v_scale", 1.0)] if fp8 else []
    a.update(kw)
    fn = B.lib().pa_prefill_attention_window_fp8 if fp8 else B.lib().pa_prefill_attention_window
    return fn(*a.values(), *scales, dt, None, None)


@pytest.mark.parametrize("call", [_decode, _chunk])
@pytest.mark.parametrize("fp8", [False, True])
def test_window_refuses(B, call, fp8):
    for kw in (dict(W=0), dict(W=-1), dict(N=-1), dict(S=-1), dict(H=0), dict(K=0), dict(D=0),
               dict(bs=0), dict(NB=0), dict(mb=0), dict(maxctx=-1), dict(H=6, K=4),
               dict(scale=float("nan")), dict(out=None), dict(q=None), dict(kc=None),
               dict(vc=None), dict(bt=None), dict(ctx=None), dict(out=ODD), dict(q=ODD),
               dict(kc=ODD), dict(vc=ODD), dict(dt=2), dict(dt=9)):
        assert call(B, fp8, **kw) == B.PA_ERR_INVALID_ARG, kw
    for kw in (dict(D=96), dict(bs=8), dict(bs=48), dict(bs=512), dict(H=34, K=2),
               dict(NB=1 << 28), dict(mb=1 << 28)):
        assert call(B, fp8, **kw) == B.PA_ERR_UNSUPPORTED, kw
    assert call(B, fp8, S=0) == B.PA_OK
    if fp8:
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert call(B, True, k_scale=bad) == B.PA_ERR_INVALID_ARG
            assert call(B, True, v_scale=bad) == B.PA_ERR_INVALID_ARG


def test_chunk_window_needs_a_positive_scale_and_offsets(B):
    assert _chunk(B, scale=0.0) == B.PA_ERR_INVALID_ARG
    assert _chunk(B, scale=-1.0) == B.PA_ERR_INVALID_ARG
    assert _chunk(B, qs=None) == B.PA_ERR_INVALID_ARG
    assert _chunk(B, T=-1) == B.PA_ERR_INVALID_ARG
    assert _chunk(B, T=0) == B.PA_OK
    assert _chunk(B, T=1 << 28) == B.PA_ERR_UNSUPPORTED
    assert _chunk(B, S=5121) == B.PA_ERR_UNSUPPORTED
    assert _chunk(B, True, S=5121) == B.PA_ERR_UNSUPPORTED


def test_window_workspace(B):
    """Partitions are counted in visible tokens, whatever the context, a
    remainder of less than half of one joining the one before; past 3 of them
    the lengths for the reduce kernel come on top."""
    f = B.pa_window_workspace_bytes
    plain = B.pa_decode_workspace_bytes
    assert f(2, 8, 2, 128, 100000, 64, 4, 0) == 0
    assert f(2, 8, 2, 128, 100000, 64, 4, 96) == 0          # 16 + 64 + 16 visible at most
    assert f(2, 8, 2, 128, 100000, 64, 4, 48) == plain(2, 8, 2, 128, 96, 48)
    assert f(2, 8, 2, 128, 50, 64, 4, 32) == plain(2, 8, 2, 128, 50, 32)
    assert f(2, 8, 2, 128, 47, 64, 4, 32) == 0               # 32 + 15
    assert f(2, 8, 2, 128, 100000, 1024, 4, 1024) == 0       # 1056 at most
    assert f(2, 8, 2, 128, 100000, 4096, 16, 1376) == plain(2, 8, 2, 128, 4128, 1376)
    assert f(2, 8, 2, 128, 100000, 4096, 16, 512) == plain(2, 8, 2, 128, 4096, 512) + 256
    assert f(3, 8, 2, 128, 100000, 128, 0, 16) == plain(3, 8, 2, 128, 144, 16) + 256
    assert f(2, 8, 2, 128, 1 << 30, 1 << 40, 1 << 40, 1 << 20) == \
        plain(2, 8, 2, 128, 1 << 30, 1 << 20) + 256         # a reach past int32 hides nothing
    for bad in ((2, 8, 2, 128, 100, 0, 4, 16), (2, 8, 2, 128, 100, 64, -1, 16),
                (-1, 8, 2, 128, 100, 64, 4, 16), (2, 8, 2, 128, 100, 64, 4, -16)):
        assert f(*bad) == 0
    need = f(2, 8, 2, 128, 128, 64, 4, 16)
    big = ctypes.c_void_p(0x40000000)
    assert _decode(B, P=16) == B.PA_ERR_WORKSPACE
    assert _decode(B, P=16, ws=big, wsb=need - 1) == B.PA_ERR_WORKSPACE
    assert _decode(B, P=16, ws=ctypes.c_void_p(0x40000010), wsb=need) == B.PA_ERR_WORKSPACE
    assert _decode(B, P=24) == B.PA_ERR_UNSUPPORTED
    many = f(2, 8, 2, 128, 4096, 1024, 4, 16)               # the lengths' region is checked too
    assert _decode(B, P=16, W=1024, maxctx=4096, mb=256, ws=big, wsb=many - 256) == \
        B.PA_ERR_WORKSPACE


def test_binding_refuses_host_tensors_and_shapes(B):
    i32, bf = torch.int32, torch.bfloat16
    z = lambda *s, dt=i32: torch.zeros(s, dtype=dt)  # noqa: E731
    q, pool = z(4, 8, 64, dt=bf), z(8, 16, 2, 64, dt=bf)
    with pytest.raises(ValueError):
        B.pa_decode_attention_window(q, q, pool, pool, z(4, 2), z(4), 32, 0.1, 16)
    with pytest.raises(ValueError):
        B.pa_decode_attention_window(q, q, pool, pool, z(3, 2), z(4), 32, 0.1, 16)
    with pytest.raises(ValueError):
        B.pa_prefill_attention_window(q, q, pool, pool, z(2, 2), z(2), z(2), 32, 0.1, 16)
    k = z(4, 2, 64, dt=bf)
    with pytest.raises(ValueError):
        B.pa_rope_and_cache(q, q, k, k, pool, pool, z(4), z(4), z(32, dt=torch.float32))
    with pytest.raises(ValueError):
        B.pa_rope_and_cache(q, q, k, k, pool, pool, z(4), z(3), z(32, dt=torch.float32))
    with pytest.raises(ValueError):
        B.pa_rope_and_cache(q, q, k, k, pool, pool, z(4), z(3, 4), z(32, dt=torch.float32),
                            axis_of_pair=z(31))
    with pytest.raises(ValueError):
        B.pa_build_step_maps(z(4, 2), z(4), z(4), z(8), z(1), 16, 8, z(5), z(9), z(9), z(9), z(4),
                             z(1))
    with pytest.raises(ValueError):
        B.pa_build_step_maps(z(4, 2), z(4), z(4), z(7), z(1), 16, 8, z(5), z(9), z(9), z(9), z(4),
                             z(1))
    # not tensors, and lists of another shape
    with pytest.raises(TypeError):
        B.pa_decode_attention_window(q, None, pool, pool, z(4, 2), z(4), 32, 0.1, 16)
    with pytest.raises(TypeError):
        B.pa_build_step_maps([[1]], z(1), z(1), z(8), z(1), 16, 8, z(2), z(9), z(9), z(9), z(1),
                             z(1))
    with pytest.raises(ValueError):
        B.pa_decode_attention_window(q[0], q[0], pool, pool, z(4, 2), z(4), 32, 0.1, 16)
    with pytest.raises(ValueError):
        B.pa_prefill_attention_window(q, q, pool, pool, z(2, 2), z(3, 1), z(2), 32, 0.1, 16)
    with pytest.raises(ValueError):
        B.pa_build_step_maps(z(4), z(4), z(4), z(8), z(1), 16, 8, z(5), z(9), z(9), z(9), z(4),
                             z(1))
