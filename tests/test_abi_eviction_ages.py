"""Host-side checks of eviction by age (no GPU)."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: checks fail first


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_96_gb300 import build
    build.build()
    from paged_kv_cache_96_gb300 import binding
    return binding


def _plan(B, **kw):
    a = dict(moves=FAKE, M=50, co=FAKE, no=FAKE, wo=FAKE, ages=FAKE, numbered=FAKE, gone=FAKE,
             bt=FAKE, mb=8, ctx=FAKE, w=FAKE, free=FAKE, cnt=FAKE, maxctx=128, limit=100,
             budget=50, sinks=4, recent=10, S=2, bs=16, N=8)
    a.update(kw)
    return B.lib().pa_plan_eviction_aged(*a.values(), None, None)


def test_aged_plan_refuses(B):
    for kw in (dict(ages=None), dict(numbered=None), dict(gone=None), dict(S=-1), dict(M=49),
               dict(mb=0), dict(bs=0), dict(N=0), dict(maxctx=-1), dict(budget=0), dict(limit=49),
               dict(sinks=-1), dict(recent=-1), dict(sinks=40, recent=11), dict(moves=None),
               dict(co=None), dict(no=None), dict(wo=None), dict(bt=None), dict(ctx=None),
               dict(w=None), dict(free=None), dict(cnt=None)):
        assert _plan(B, **kw) == B.PA_ERR_INVALID_ARG, kw
    for kw in (dict(bs=24), dict(N=1 << 28), dict(mb=1 << 28), dict(M=(1 << 29) + 1)):
        assert _plan(B, **kw) == B.PA_ERR_UNSUPPORTED, kw


def test_contexts_whose_counting_would_pass_32_bits_are_refused(B):
    """Places are counted in steps of up to 4,096 past the longest context."""
    top = (1 << 31) - 1
    for bs, mb in ((16, (1 << 27) - 1), (1, top), (1, top - 65535)):
        big = dict(bs=bs, mb=mb, N=mb, maxctx=top)
        assert _plan(B, **big) == B.PA_ERR_UNSUPPORTED, big
        a = dict(moves=FAKE, M=50, co=FAKE, no=FAKE, wo=FAKE, bt=FAKE, mb=8, ctx=FAKE, w=FAKE,
                 free=FAKE, cnt=FAKE, maxctx=128, limit=100, budget=50, sinks=4, recent=10, S=2,
                 bs=16, N=8)
        a.update(big)
        assert B.lib().pa_plan_eviction(*a.values(), None, None) == B.PA_ERR_UNSUPPORTED, big


def test_ages_are_keywords_of_the_plan(B):
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    w = torch.zeros((8, 16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.pa_plan_eviction(z(4, 9, 2), z(4), z(1), w, z(4, 2), z(4), w, z(8), z(1), 32, 16, 8,
                           arrivals=z(8, 16), numbered_lens=z(4), evicted=z(4))
