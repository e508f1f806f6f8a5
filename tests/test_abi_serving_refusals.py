"""Host-side refusals of the serving-step operators beside those of
test_abi_serving_ops.py: a status or an exception before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

from test_abi_serving_ops import B, _chunk, _decode, _rope  # noqa: F401


@pytest.mark.parametrize("call", [_decode, _chunk])
def test_window_refuses_scales_whose_product_overflows(B, call):  # noqa: F811
    assert call(B, scale=3e38) == B.PA_ERR_INVALID_ARG           # times log2(e)
    assert call(B, True, scale=1e30, k_scale=1e9) == B.PA_ERR_INVALID_ARG
    assert call(B, S=0, scale=2e38) == B.PA_OK
    assert call(B, True, S=0, scale=1e30, k_scale=1e8) == B.PA_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_in_place_refuses_keys_and_values_of_the_query(B, fp8):  # noqa: F811
    """The rotated query over rows that keys or values are still read from."""
    q, other = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x40000000)
    head = ctypes.c_void_p(0x100000 + 2 * 128)              # the query's second head
    next_row = ctypes.c_void_p(0x100000 + 2 * 1024)
    for k, v in ((q, other), (other, q), (q, q), (head, other), (other, head)):
        for T in (1, 4):
            assert _rope(B, fp8, q=q, qo=q, k=k, v=v, ks=1024, vs=1024, T=T) == \
                B.PA_ERR_INVALID_ARG
        assert _rope(B, fp8, q=q, qo=q, k=k, v=v) == B.PA_ERR_INVALID_ARG
    # a key in the query's next row (of several tokens)
    assert _rope(B, fp8, q=q, qo=q, k=next_row, v=other, ks=1024) == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [16.0, 16.9, "16", None, np.float32(16), torch.tensor(16.0)])
def test_binding_takes_integers_only(B, bad):  # noqa: F811
    """Nothing is cut to an integer or read from a text, as in the calls through ctypes."""
    f = B.pa_window_workspace_bytes
    good = f(2, 8, 2, 128, 4096, 1024, 4, 256)
    assert good > 0 and f(2, 8, 2, 128, np.int64(4096), np.int32(1024), np.uint8(4), 256) == good
    for i in range(8):
        with pytest.raises((TypeError, ctypes.ArgumentError)):
            f(*[bad if i == k else x for k, x in enumerate((2, 8, 2, 128, 4096, 1024, 4, 256))])
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for size, blocks in ((bad, 8), (16, bad)):
        with pytest.raises(TypeError):
            B.pa_build_step_maps(z(4, 2), z(4), z(4), z(8), z(1), size, blocks, z(5), z(9), z(9),
                                 z(9), z(4), z(1))


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_refuses_outputs_over_its_queries(B, fp8):  # noqa: F811
    q = 0x100000
    size = 2 * 9 * 8 * 128                                   # of _chunk's 9 rows
    for out in (q, q + 16, q + size - 16, q - size + 16):
        assert _chunk(B, fp8, out=ctypes.c_void_p(out), q=ctypes.c_void_p(q)) == \
            B.PA_ERR_INVALID_ARG
