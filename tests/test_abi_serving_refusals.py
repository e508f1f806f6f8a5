"""Host-side refusals of the serving-step operators beside those of
test_abi_serving_ops.py: a status or an exception before anything is launched."""
import ctypes

import pytest

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
