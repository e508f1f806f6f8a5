"""Decode attention that accumulates weights against the definition in 64 bits.

Pools hold NaN past every context, and so do the weights that a call has no business
reading."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import context_refs as C  # noqa: E402
from operator_refs import assert_within  # noqa: E402
from test_gpu_sparse_decode import IDS, SCALE, TYPES, i32  # noqa: E402


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


class Case:
    def __init__(self, ctx, weighted, H, K, D, bs, dtype, fp8, seed=0, slack=0):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.fp8, self.bs = dtype, fp8, bs
        self.ctx, self.weighted = np.asarray(ctx), np.asarray(weighted)
        blocks = -(-self.ctx // bs)
        N, MB = int(blocks.sum()) + 3, max(1, int(blocks.max()))
        ids = r.permutation(N)
        self.tables = np.full((len(ctx), MB), N + 5, dtype=np.int32)
        live = np.zeros((N, bs), dtype=bool)
        old = np.zeros((N, bs), dtype=bool)
        at = 0
        for s, n in enumerate(blocks):
            self.tables[s, :n] = ids[at:at + n]
            at += n
            p = np.arange(self.ctx[s])
            live[self.tables[s, p // bs], p % bs] = True
            p = p[:self.weighted[s]]
            old[self.tables[s, p // bs], p % bs] = True
        shape = (N, bs, K, D)
        k, v = (torch.randn(shape, generator=g) for _ in range(2))
        hide = torch.as_tensor(~live)[..., None, None].expand(shape)
        if fp8:
            self.kc, self.vc = ((x / SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)
                                .view(torch.uint8).masked_fill(hide, 0x7F).cuda()
                                for x in (k, v))
        else:
            self.kc, self.vc = (x.to(dtype).masked_fill(hide, float("nan")).cuda()
                                for x in (k, v))
        w = torch.rand((N, bs), generator=g) * 3
        self.weights = w.masked_fill(torch.as_tensor(~old), float("nan")).cuda()
        self.live, self.old = live, old
        self.q = torch.randn((len(ctx), H, D), generator=g).to(dtype).cuda()
        self.out = torch.full_like(self.q, 7.0)
        self.weights_out = torch.full_like(self.weights, -5.0)
        self.max_ctx = int(self.ctx.max()) + slack
        self.scale, self.kv = D ** -0.5, SCALE if fp8 else 1.0
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def workspace(self, B, P):
        S, H, D = self.q.shape
        n = B.pa_weights_workspace_bytes(S, H, self.kc.shape[2], D, self.max_ctx, P)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where it may be
        ws[:1 << 20] = 0
        return ws

    def run(self, B, P=0, ws=None, weights=None, weights_out=None, **kw):
        ws = self.workspace(B, P) if ws is None else ws
        args = [i32(x) for x in (self.tables, self.ctx, self.weighted)]
        torch.cuda.synchronize()
        B.pa_decode_attention_weights(
            self.out, self.weights_out if weights_out is None else weights_out, self.q, self.kc,
            self.vc, self.weights if weights is None else weights, *args, self.max_ctx,
            self.scale, ws, P, k_scale=self.kv, v_scale=self.kv, error_word=self.err, **kw)
        torch.cuda.synchronize()

    def want(self):
        kc, vc = (C.pool_values(x, self.kv) for x in (self.kc, self.vc))
        w = np.where(self.old, self.weights.cpu().numpy(), 0)
        return C.weights_attention(self.q, kc, vc, w, self.tables, self.ctx, self.weighted,
                                   self.scale, self.dtype,
                                   torch.float16 if self.fp8 else self.dtype)

    def check(self, weights_out=None, what=""):
        assert int(self.err.item()) == 0
        got = (self.weights_out if weights_out is None else weights_out).double().cpu().numpy()
        want, tol, new, new_tol = self.want()
        assert_within(self.out, want, tol, what)
        far = np.abs(got - new)[self.live]
        assert np.isfinite(far).all()
        worst = (far / new_tol[self.live]).max() if far.size else 0
        assert worst <= 1, f"{what}: weights {worst:.2f}x their bound"
        # each head's weights add up to one
        return got


SHAPES = [
    # H, K, D, bs, contexts, weighted
    (4, 4, 64, 16, [1, 2, 15, 16, 17, 500], [0, 1, 15, 15, 0, 499]),
    (8, 2, 128, 16, [33, 0, 1000, 64], [33, 0, 0, 10]),
    (16, 1, 64, 32, [700, 31, 1], [699, 40, 1]),       # more weighted than there are
    (10, 2, 128, 64, [300, 65], [299, 0]),
    (3, 1, 128, 16, [1537], [1536]),
    (14, 2, 64, 256, [255, 900], [0, 899]),
    (9, 1, 64, 128, [129, 515], [128, 500]),
    (8, 8, 128, 16, [333, 15], [332, 14]),
    (24, 8, 128, 16, [260], [0]),
]


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("H,K,D,bs,ctx,weighted", SHAPES)
def test_weights_match_the_definition(B, dtype, fp8, H, K, D, bs, ctx, weighted):
    c = Case(ctx, weighted, H, K, D, bs, dtype, fp8, seed=H * D + bs, slack=D)
    for P in (0, 16, 64, 256):
        c.out.fill_(7.0)
        c.weights_out.fill_(-5.0)
        c.run(B, P)
        got = c.check(what=f"partition {P}")
        assert (got[~c.live] == -5.0).all()            # no position of the batch


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_in_place_repeat_and_replay(B, fp8):
    c = Case([400, 33, 1200], [399, 0, 1199], 8, 2, 128, 16, torch.bfloat16, fp8, seed=2)
    c.run(B, 128)
    first, out = c.weights_out.clone(), c.out.clone()
    both = c.weights.clone()
    c.run(B, 128, weights=both, weights_out=both, stream=torch.cuda.Stream())
    live = torch.as_tensor(c.live).cuda()
    assert torch.equal(both[live], first[live]) and torch.equal(c.out, out)
    c.check(weights_out=both)
    ws = c.workspace(B, 128)
    args = [i32(x) for x in (c.tables, c.ctx, c.weighted)]
    call = lambda: B.pa_decode_attention_weights(  # noqa: E731
        c.out, c.weights_out, c.q, c.kc, c.vc, c.weights, *args, c.max_ctx, c.scale, ws, 128,
        k_scale=c.kv, v_scale=c.kv, error_word=c.err)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        c.out.zero_(), c.weights_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.weights_out[live], first[live]) and torch.equal(c.out, out)


def test_weights_of_many_sequences(B):
    """More sequences than the default rings leave room for, most of one token."""
    r = np.random.default_rng(7)
    ctx = r.integers(0, 3, size=9000)
    ctx[[5, 4000, 8999]] = [300, 0, 777]
    c = Case(ctx, np.maximum(ctx - 1, 0), 2, 1, 64, 16, torch.float16, False, seed=3)
    c.run(B, 256)
    c.check()


def test_weights_flag_what_is_out_of_range(B):
    from paged_kv_cache_96_gb300 import binding as L
    c = Case([100, 90], [99, 89], 4, 1, 64, 16, torch.float16, False, seed=6)
    want, tol, new, new_tol = c.want()
    keep = c.tables.copy()
    for bad in (-2, 1 << 25):
        c.tables = keep.copy()
        c.tables[0, 2] = bad
        c.err.zero_()
        c.weights_out.fill_(-5.0)
        c.run(B, 32)
        assert int(c.err.item()) == L.DEVERR_BLOCK_RANGE
        got = c.weights_out.double().cpu().numpy()
        assert (got[keep[0, 2]] == -5.0).all()
        p = np.arange(90)
        at = (keep[1][p // 16], p % 16)
        assert (np.abs(got[at] - new[at]) <= new_tol[at]).all()
        assert np.isfinite(got[keep[0, 1]]).all()
    c.tables, c.max_ctx = keep, 64
    c.err.zero_()
    c.run(B, 32)                                       # contexts clipped to 64
    assert int(c.err.item()) == L.DEVERR_CONTEXT_RANGE
    c.err.zero_()
    short = Case([64, 64], [64, 64], 4, 1, 64, 16, torch.float16, False)
    short.tables, short.kc, short.vc, short.q = keep, c.kc, c.vc, c.q
    want, tol, _, _ = C.weights_attention(c.q, *(C.pool_values(x, 1.0) for x in (c.kc, c.vc)),
                                          np.zeros(c.weights.shape), keep, [64, 64], [0, 0],
                                          c.scale, c.dtype, c.dtype)
    assert_within(c.out, want, tol)


def test_special_scores(B):
    """A key that is not a number makes its sequence's weights so and no other's; keys of
    -inf have a weight of 0."""
    c = Case([40, 40, 40], [0, 0, 0], 4, 1, 64, 16, torch.bfloat16, False, seed=12)
    c.q.abs_()
    t = c.tables
    c.kc[t[0, 1], 3, 0, 0] = float("nan")
    c.kc[t[1, 2], 0, 0, 0] = -float("inf")
    c.run(B, 16)
    assert int(c.err.item()) == 0
    p = np.arange(40)
    got = [c.weights_out.cpu().numpy()[t[s][p // 16], p % 16] for s in range(3)]
    assert np.isnan(got[0]).all() and np.isfinite(got[1]).all() and np.isfinite(got[2]).all()
    assert got[1][32] == 0 and abs(got[1].sum() - 4) < 1e-5 and abs(got[2].sum() - 4) < 1e-5


def test_two_steps_on_two_streams(B):
    """Two batches with a workspace each, at the same time."""
    cs = [Case([900, 100], [899, 99], 16, 2, 128, 16, torch.bfloat16, False, seed=s)
          for s in (20, 21)]
    ws = [c.workspace(B, 64) for c in cs]
    args = [[i32(x) for x in (c.tables, c.ctx, c.weighted)] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, w, a, s in zip(cs, ws, args, streams):
            B.pa_decode_attention_weights(c.out, c.weights_out, c.q, c.kc, c.vc, c.weights, *a,
                                          c.max_ctx, c.scale, w, 64, error_word=c.err, stream=s)
    torch.cuda.synchronize()
    for c in cs:
        c.check()


@pytest.mark.parametrize("P", [0, 64])
def test_no_token_at_all(B, P):
    """Empty contexts, and a longest context of 0."""
    c = Case([0, 0, 0], [0, 5, -3], 4, 2, 64, 16, torch.float16, False, seed=1, slack=100)
    c.run(B, P)
    c.check()
    c.max_ctx = 0
    c.out.fill_(7.0)
    c.run(B, P)
    c.check()
    assert not c.out.any() and (c.weights_out == -5.0).all()


def test_scores_past_32_bits(B):
    """A longest context that puts the second sequence's scores past 4 GB."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    c = Case([33, 700], [0, 699], 128, 8, 64, 16, torch.bfloat16, False, seed=4)
    c.max_ctx = 10_000_000
    c.tables = np.concatenate([c.tables, np.full((2, 625_000 - c.tables.shape[1]), -1,
                                                 dtype=np.int32)], 1)
    for P in (0, 512):
        c.out.fill_(7.0)
        c.weights_out.fill_(-5.0)
        c.run(B, P)
        c.check(what=f"partition {P}")


def test_one_long_sequence_among_many(B):
    """Shares of a batch in which one context holds most tokens, and its partials pass
    what the pass merges itself."""
    ctx = [3] * 40 + [30000] + [1] * 30
    c = Case(ctx, [2] * 40 + [29999] + [0] * 30, 8, 8, 64, 32, torch.bfloat16, True, seed=5)
    for P in (0, 16, 256):
        c.out.fill_(7.0)
        c.run(B, P)
        c.check(what=f"partition {P}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P", [0, 32])
def test_a_wait_runs_out_and_the_next_call_answers(B, P, fp8):
    c = Case([500, 90, 333], [499, 0, 332], 8, 2, 128, 16, torch.bfloat16, fp8, seed=6)
    ws = c.workspace(B, P)
    try:
        B.pa_set_stage_wait_limit_ns(2_000_000)
        B.pa_debug_withhold_first_fill(True)
        c.run(B, P, ws)
    finally:
        B.pa_debug_withhold_first_fill(False)
        B.pa_set_stage_wait_limit_ns(0)
    assert int(c.err.item()) == B.DEVERR_TIMEOUT
    c.err.zero_()
    c.run(B, P, ws)
    c.check()


def test_one_workspace_for_calls_with_and_without_partitions(B):
    """A call on whole contexts leaves the arrival counters of the others at zero."""
    c = Case([900, 333, 16], [899, 0, 15], 16, 2, 128, 16, torch.bfloat16, False, seed=9)
    ws = max((c.workspace(B, P) for P in (0, 32, 256)), key=lambda w: w.numel())
    for P in (0, 32, 0, 256, 0, 32):
        c.out.fill_(7.0)
        c.weights_out.fill_(-5.0)
        c.run(B, P, ws)
        c.check(what=f"partition {P}")
        assert not ws[:1 << 20].any()
