"""Edges of the long-context operators."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_block_selection import Bounds  # noqa: E402
from test_gpu_sparse_decode import IDS, TYPES, Case as Lists  # noqa: E402
from test_gpu_weights_decode import SHAPES, Case as Weights  # noqa: E402


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


def kernels_of(call):
    """Launches of a call, as a captured graph holds them."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t()
    status = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(
        ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n))
    assert status == 0
    return n.value


@pytest.mark.parametrize("top_k,parts", [(4, 2), (6, 3), (8, 4), (9, 5), (10, 4), (11, 6)])
def test_rows_of_more_than_four_partials_go_to_the_reduce_kernel(B, top_k, parts):
    """Lists in shares of their own, of 2 tiles (10 tiles: of 3); a last tile by itself is a
    share too."""
    ctx = np.array([400, 333])
    c = Lists(ctx, [0, 1], ctx - 1, 4, 1, 64, 16, top_k, torch.bfloat16, False, seed=top_k)
    ws = c.workspace(B, 32)
    args = [torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()
            for a in (c.tables, c.seq, c.pos, c.chosen)]
    call = lambda: B.pa_decode_attention_sparse(  # noqa: E731
        c.out, c.q, c.kc, c.vc, *args, c.scale, 32, ws, error_word=c.err)
    assert kernels_of(call) == (2 if parts > 4 else 1)
    c.out.fill_(7.0)
    c.run(B, 32, ws)
    c.check()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("H,K,D,bs,ctx", [x[:5] for x in SHAPES])
def test_a_steps_weights_add_up_to_the_heads(B, dtype, fp8, H, K, D, bs, ctx):
    """Each head's weights over a context have a sum of 1, however the scores are rounded:
    what is counted is the sums' own error (a term for every second token of a lane, every
    head and a few partials), that of three exponentials, and their arguments' for scores
    of at most 32."""
    c = Weights(ctx, np.zeros(len(ctx), dtype=int), H, K, D, bs, dtype, fp8, seed=H * D)
    for P in (0, 16, 256):
        c.weights_out.fill_(-5.0)
        c.run(B, P)
        assert int(c.err.item()) == 0
        got = c.weights_out.double().cpu().numpy()
        for s, n in enumerate(ctx):
            p = np.arange(n)
            tol = H * ((2 * -(-n // 16) + H + 16 + 128) * 2.0 ** -24 + 3 * 2.0 ** -21)
            total = got[c.tables[s][p // bs], p % bs].sum()
            assert abs(total - (H if n else 0)) <= tol, (s, n, P)
