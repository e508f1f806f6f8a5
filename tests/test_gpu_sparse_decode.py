"""Attention over lists of blocks against the definition in 64 bits.

Pools hold NaN wherever no row of a KV head sees a token, and table entries of blocks
that no list names point outside the pool."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import context_refs as C  # noqa: E402
from operator_refs import assert_within  # noqa: E402

SCALE = 0.02
TYPES = [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
         (torch.float16, True)]
IDS = ["bf16", "f16", "bf16-fp8", "f16-fp8"]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Case:
    def __init__(self, ctx, seq, pos, H, K, D, bs, top_k, dtype, fp8, seed=0, chosen=None,
                 poison=True):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.fp8, self.bs = dtype, fp8, bs
        self.seq, self.pos = np.asarray(seq), np.asarray(pos)
        ctx = np.asarray(ctx)
        T = len(seq)
        blocks = -(-ctx // bs)
        N, MB = int(blocks.sum()) + 3, max(1, int(blocks.max()))
        ids = r.permutation(N)
        full = np.zeros((len(ctx), MB), dtype=np.int32)
        at = 0
        for s, n in enumerate(blocks):
            full[s, :n] = ids[at:at + n]
            at += n
        if chosen is None:
            chosen = np.full((T, K, top_k), -1, dtype=np.int32)
            for t in range(T):
                if seq[t] < 0:
                    chosen[t] = r.integers(-3, 1000, size=(K, top_k))  # never looked at
                    continue
                have = pos[t] // bs + 1
                for h in range(K):
                    n = min(have, top_k)
                    pick = r.permutation(have)[:n]
                    pick[0] = have - 1
                    chosen[t, h, :n] = np.unique(np.concatenate([pick, pick[:1]]))[:n] \
                        if len(np.unique(pick)) == n else r.permutation(have)[:n]
        self.chosen = np.asarray(chosen)
        self.tables = np.full_like(full, N + 5)
        live = np.zeros((N, bs, K), dtype=bool)
        for t in range(T):
            if seq[t] < 0:
                continue
            for h in range(K):
                n = min(top_k, pos[t] // bs + 1)
                for b in self.chosen[t, h, :n]:
                    if 0 <= b <= pos[t] // bs:
                        self.tables[seq[t], b] = full[seq[t], b]
                        seen = np.arange(bs) + b * bs <= pos[t]
                        live[full[seq[t], b], :, h] |= seen
        shape = (N, bs, K, D)
        k, v = (torch.randn(shape, generator=g) for _ in range(2))
        hide = torch.as_tensor(~live if poison else live & False)[..., None].expand(shape)
        if fp8:
            self.kc, self.vc = ((x / SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)
                                .view(torch.uint8).masked_fill(hide, 0x7F).cuda()
                                for x in (k, v))
        else:
            self.kc, self.vc = (x.to(dtype).masked_fill(hide, float("nan")).cuda()
                                for x in (k, v))
        self.q = torch.randn((T, H, D), generator=g).to(dtype).cuda()
        self.out = torch.full_like(self.q, 7.0)
        self.scale, self.kv = D ** -0.5, SCALE if fp8 else 1.0
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def workspace(self, B, P):
        T, H, D = self.q.shape
        n = B.pa_sparse_workspace_bytes(T, H, self.kc.shape[2], D, self.chosen.shape[2], self.bs,
                                        P)
        return torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None

    def run(self, B, P=0, ws=None, **kw):
        ws = self.workspace(B, P) if ws is None else ws
        args = [i32(x) for x in (self.tables, self.seq, self.pos, self.chosen)]
        torch.cuda.synchronize()
        B.pa_decode_attention_sparse(self.out, self.q, self.kc, self.vc, *args, self.scale, P, ws,
                                     k_scale=self.kv, v_scale=self.kv, error_word=self.err, **kw)
        torch.cuda.synchronize()
        return self.out.clone()

    def want(self):
        kc, vc = (C.pool_values(x, self.kv) for x in (self.kc, self.vc))
        return C.sparse_attention(self.q, kc, vc, self.tables, self.seq, self.pos, self.chosen,
                                  self.scale, self.dtype,
                                  torch.float16 if self.fp8 else self.dtype)

    def check(self, what=""):
        assert int(self.err.item()) == 0
        want, tol = self.want()
        assert_within(self.out, want, tol, what)


LISTS = [
    # H, K, D, bs, top_k, contexts
    (4, 4, 64, 16, 8, [1, 2, 16, 17, 500]),
    (8, 2, 128, 16, 3, [1, 33, 47, 48, 49, 100]),
    (16, 1, 64, 32, 5, [31, 32, 33, 200, 1000]),
    (10, 2, 128, 64, 4, [63, 64, 65, 300, 301]),
    (3, 1, 128, 16, 40, [700, 640, 641]),
    (32, 2, 128, 256, 3, [255, 256, 900, 1500]),
    (9, 1, 64, 128, 2, [1, 129, 515]),
    (8, 8, 128, 16, 1, [1, 15, 333]),
]


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("H,K,D,bs,top_k,ctx", LISTS)
def test_sparse_matches_the_definition(B, dtype, fp8, H, K, D, bs, top_k, ctx):
    c = Case(ctx, np.arange(len(ctx)), np.asarray(ctx) - 1, H, K, D, bs, top_k, dtype, fp8,
             seed=H * D + bs)
    for P in (0, 16, 48, 256):
        c.out.fill_(7.0)
        c.run(B, P)
        c.check(f"partition {P}")


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_rows_of_one_sequence_padding_and_long_lists(B, dtype, fp8):
    """Several rows of a sequence, padding rows between, and lists of more than 32 tiles
    a warp in one partition and in many."""
    seq = np.array([0, 0, -1, 1, 0, 1, -7])
    pos = np.array([3999, 3998, -1, 5000, 17, 100, 5])
    c = Case([4000, 5001], seq, pos, 8, 2, 64, 16, 200, dtype, fp8, seed=5)
    for P in (0, 128, 512, 1024):
        c.out.fill_(7.0)
        c.run(B, P)
        c.check(f"partition {P}")
    assert not c.out[[2, 6]].any()


def test_many_rows(B):
    """More units than CTAs: rows of different list lengths side by side."""
    r = np.random.default_rng(3)
    ctx = r.integers(1, 400, size=90)
    c = Case(ctx, np.arange(90), ctx - 1, 16, 8, 64, 16, 12, torch.bfloat16, False, seed=4)
    ws = c.workspace(B, 64)
    for P in (0, 64):
        c.run(B, P, ws)
        c.check(f"partition {P}")


def lists(rows, top_k):
    out = np.full((len(rows), 1, top_k), -1, dtype=np.int32)
    for t, x in enumerate(rows):
        out[t, 0, :len(x)] = x
    return out


@pytest.mark.parametrize("P", [0, 16, 32, 64])
def test_lists_with_holes_repeats_and_nothing(B, P):
    ctx = [200] * 6
    chosen = lists([[3, -1, 12, -1, 0, -5], [5, 5, 12], [], [-1, -1, -1, -1, -1, 12],
                    [12, 1, 0, 7, 7, 7], [-9, 4]], 6)
    c = Case(ctx, np.arange(6), np.full(6, 199), 4, 1, 64, 16, 6, torch.float16, False, seed=8,
             chosen=chosen)
    c.run(B, P)
    c.check()
    assert not c.out[2].any()


@pytest.mark.parametrize("P", [0, 32])
def test_what_a_row_sees_counts_and_nothing_else(B, P):
    """An infinity, a NaN and keys of -inf in listed blocks, and rows without any."""
    chosen = lists([[0, 3, 5], [1, 3, 5], [2, 2, 2], [4, -1, -1], [-1, -1, -1], [0, 1, 5]], 6)
    c = Case([96] * 6, np.arange(6), np.full(6, 95), 4, 1, 64, 16, 6, torch.bfloat16, False,
             seed=9, chosen=chosen)
    t = c.tables
    c.q.abs_()
    c.vc[t[0, 3], 2, 0, 7] = float("inf")           # row 0: one column infinite
    c.kc[t[1, 1], 4, 0, 0] = float("nan")           # row 1: not a number
    c.kc[t[2, 2], :, 0, 0] = -float("inf")          # row 2: no weight anywhere
    c.kc[t[5, 1], :, 0, 0] = -float("inf")          # row 5: no weight in one block
    got = c.run(B, P).float()
    assert int(c.err.item()) == 0
    assert (got[0, :, 7] == float("inf")).all()
    assert torch.isfinite(got[0, :, :7]).all() and torch.isfinite(got[0, :, 8:]).all()
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
    assert torch.isfinite(got[3]).all() and (got[3] != 0).any()
    assert (got[4] == 0).all()
    clean = Case([96] * 6, np.arange(6), np.full(6, 95), 4, 1, 64, 16, 6, torch.bfloat16, False,
                 seed=9, chosen=lists([[0], [1], [2], [4], [], [0, 5]], 6))
    clean.kc, clean.vc, clean.q, clean.tables = c.kc, c.vc, c.q, c.tables
    want, tol = clean.want()
    far = np.abs(got[5].double().cpu().numpy() - want[5])
    assert (far <= tol[5]).all()


def test_sparse_flags_what_is_out_of_range(B):
    from paged_kv_cache_96_gb300 import binding as L
    base = [[0, 3, 5]] * 3
    for change, flag in ((dict(entry=6), L.DEVERR_CONTEXT_RANGE),
                         (dict(entry=1 << 29), L.DEVERR_CONTEXT_RANGE),
                         (dict(seq=3), L.DEVERR_TOKEN_RANGE), (dict(pos=-1), L.DEVERR_TOKEN_RANGE),
                         (dict(pos=96), L.DEVERR_TOKEN_RANGE),
                         (dict(table=-1), L.DEVERR_BLOCK_RANGE),
                         (dict(table=1 << 20), L.DEVERR_BLOCK_RANGE)):
        for P in (0, 16):
            c = Case([96] * 3, np.arange(3), np.full(3, 95), 4, 1, 64, 16, 6, torch.float16,
                     False, seed=9, chosen=lists(base, 6))
            want, tol = c.want()
            if "entry" in change:
                c.chosen[1, 0, 1] = change["entry"]
            if "seq" in change:
                c.seq[1] = change["seq"]
            if "pos" in change:
                c.pos[1] = change["pos"]
            if "table" in change:
                c.tables[1, 3] = change["table"]
            got = c.run(B, P)
            assert int(c.err.item()) == flag, change
            rest = [0, 2]
            assert_within(got[rest], want[rest], tol[rest])
            if "seq" in change or "pos" in change:
                assert not got[1].any()
            else:                                   # as without the entry
                c.chosen[1, 0, 1] = -1
                c.tables[1, 3] = 0
                want, tol = c.want()
                assert_within(got[1:2], want[1:2], tol[1:2])


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_over_all_blocks_is_decode(B, fp8):
    """Lists of every block against windowed decode with a window past the context, and
    the same bits in a second call, on another stream and from a replayed graph."""
    ctx = np.array([700, 33, 512])
    every = np.full((3, 2, 44), -1, dtype=np.int32)
    for t in range(3):
        n = -(-ctx[t] // 16)
        every[t, :, :n] = np.arange(n)
    c = Case(ctx, np.arange(3), ctx - 1, 8, 2, 128, 16, 44, torch.bfloat16, fp8, seed=1,
             chosen=every)
    a = c.run(B, 128)
    c.check()
    side = torch.cuda.Stream()
    assert torch.equal(a, c.run(B, 128, stream=side))
    ws = c.workspace(B, 128)
    args = [i32(x) for x in (c.tables, c.seq, c.pos, c.chosen)]
    call = lambda: B.pa_decode_attention_sparse(c.out, c.q, c.kc, c.vc, *args, c.scale, 128, ws,  # noqa: E731
                                                k_scale=c.kv, v_scale=c.kv, error_word=c.err)
    graph = torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        c.out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, c.out)
    dense = torch.empty_like(c.out)
    B.pa_decode_attention_window(dense, c.q, c.kc, c.vc, args[0], i32(ctx), 700, c.scale, 1 << 20,
                                 k_scale=c.kv, v_scale=c.kv, error_word=c.err)
    torch.cuda.synchronize()
    _, tol = c.want()
    assert_within(a, dense.double().cpu().numpy(), 2 * tol)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P", [0, 32])
def test_a_wait_runs_out_and_the_next_call_answers(B, P, fp8):
    ctx = np.array([500, 90, 333])
    c = Case(ctx, np.arange(3), ctx - 1, 8, 2, 128, 16, 9, torch.bfloat16, fp8, seed=6)
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


def test_graphs_that_share_a_workspace(B):
    """Two captured calls of different sizes over one workspace, replayed in turn."""
    cs = [Case([700, 33, 512], [0, 1, 2], np.array([699, 32, 511]), 8, 2, 128, 16, 40,
               torch.bfloat16, False, seed=1),
          Case([900], [0, 0], np.array([899, 898]), 16, 1, 64, 32, 12, torch.float16, True,
               seed=2)]
    ws = max((c.workspace(B, 64) for c in cs), key=lambda w: w.numel())
    args = [[i32(x) for x in (c.tables, c.seq, c.pos, c.chosen)] for c in cs]
    graphs = []
    for c, a in zip(cs, args):
        call = lambda: B.pa_decode_attention_sparse(  # noqa: E731
            c.out, c.q, c.kc, c.vc, *a, c.scale, 64, ws, k_scale=c.kv, v_scale=c.kv,
            error_word=c.err)
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(3):
        for c in cs:
            c.out.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c in cs:
            c.check()
