"""Edges of the long-context operators."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_block_selection import Bounds  # noqa: E402


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


@pytest.mark.parametrize("ctx,rows,top_k", [
    (2000, 1, 9),                              # one warp selects
    (12000, 1, 40),                            # a cluster of CTAs
    (12000, 700, 40),                          # one CTA a row, by all of its warps
])
def test_scores_of_either_zero_are_equal(B, ctx, rows, top_k):
    """Bounds with a scale of 0 beside codes that are not, as a cache filled elsewhere may
    bring them: a score of -0 is that of +0, and the lower block goes first."""
    x = Bounds([ctx], 1, 64, 16, seed=3)
    x.codes[:] = np.minimum(-1, -np.abs(x.codes.astype(int))).astype(np.int8)  # scores below 0
    t = x.tables[0]
    x.scales[t[10:60]] = 0                     # -0
    x.codes[t[40:90:2]] = 0                    # +0, of a scale that is 0 or not
    q = torch.rand((rows, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    got = x.select(B, q, np.zeros(rows, dtype=int), np.full(rows, ctx - 1), top_k, 1, 1)
    assert int(x.err.item()) == 0
    last = -(-ctx // 16) - 1
    assert got[0, 0].tolist() == [0] + list(range(10, 10 + top_k - 2)) + [last]
    assert (got == got[0]).all()
