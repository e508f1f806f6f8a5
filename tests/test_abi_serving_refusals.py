"""Host-side refusals of the serving-step operators beside those of
test_abi_serving_ops.py: a status or an exception before anything is launched."""
import pytest

from test_abi_serving_ops import B, _chunk, _decode  # noqa: F401


@pytest.mark.parametrize("call", [_decode, _chunk])
def test_window_refuses_scales_whose_product_overflows(B, call):  # noqa: F811
    assert call(B, scale=3e38) == B.PA_ERR_INVALID_ARG           # times log2(e)
    assert call(B, True, scale=1e30, k_scale=1e9) == B.PA_ERR_INVALID_ARG
    assert call(B, S=0, scale=2e38) == B.PA_OK
    assert call(B, True, S=0, scale=1e30, k_scale=1e8) == B.PA_OK
