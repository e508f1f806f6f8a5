"""Eviction plans and token moves against their definitions, for equality."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import context_refs as C  # noqa: E402


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Plan:
    def __init__(self, ctx, bs, limit, budget, sinks, recent, seed=0, levels=0, spare=5):
        r = np.random.default_rng(seed)
        self.ctx, self.bs = np.asarray(ctx), bs
        self.rule = (limit, budget, sinks, recent)
        blocks = -(-self.ctx // bs)
        self.N, MB = int(blocks.sum()) + spare, max(1, int(blocks.max()))
        ids = r.permutation(self.N)
        self.tables = np.full((len(ctx), MB), -3, dtype=np.int32)   # entries never looked at
        at = 0
        for s, n in enumerate(blocks):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.free = np.full(self.N, -7, dtype=np.int32)
        self.free[:spare] = ids[at:]
        self.count = spare
        w = np.exp(r.normal(size=(self.N, bs))) if levels == 0 else \
            r.integers(0, levels, size=(self.N, bs)) / 4
        self.weights = w.astype(np.float32)
        self.max_ctx = int(self.ctx.max())
        self.capacity = max(1, min(budget, self.max_ctx - budget)) + seed % 3
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, B, in_place=False, **kw):
        w, ctx, count = torch.as_tensor(self.weights).cuda(), i32(self.ctx), i32([self.count])
        w_out = w if in_place else torch.full_like(w, -2.0)
        ctx_out = ctx if in_place else torch.full_like(ctx, -2)
        count_out = count if in_place else i32([-2])
        moves = torch.full((len(self.ctx), self.capacity, 2), 55, dtype=torch.int32,
                           device="cuda")
        free, tables = i32(self.free), i32(self.tables)
        torch.cuda.synchronize()
        B.pa_plan_eviction(moves, ctx_out, count_out, w_out, tables, ctx, w, free, count,
                           kw.pop("max_ctx", self.max_ctx), *self.rule, error_word=self.err, **kw)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in (moves, ctx_out, free, count_out, w_out)]

    def want(self):
        return C.plan_eviction(self.tables, self.ctx, self.weights, self.free, self.count, self.bs,
                               *self.rule, self.capacity)

    def check(self, B, in_place=False, **kw):
        got, want = self.run(B, in_place, **kw), self.want()
        assert int(self.err.item()) == 0
        for name, g, w in zip(("moves", "lengths", "free", "count"), got, want):
            assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), name
        new = want[4]
        if in_place:
            stays = np.ones(new.shape, dtype=bool)
            # (a place that a token has left is as it was)
        else:
            stays = np.zeros(new.shape, dtype=bool)
            for s, n in enumerate(want[1]):
                p = np.arange(n)
                stays[self.tables[s, p // self.bs], p % self.bs] = True
            assert (got[4][~stays] == -2.0).all()
        assert np.array_equal(got[4][stays], new[stays])
        return got


RULES = [
    # contexts, block, limit, budget, sinks, recent
    ([1, 50, 51, 100, 101, 500], 16, 100, 50, 4, 10),
    ([300, 17, 0, 301], 16, 300, 300, 0, 0),               # one token goes
    ([64, 65, 128, 129], 64, 64, 64, 1, 63),               # nothing is chosen by weight
    ([900, 1000, 31], 32, 40, 33, 0, 1),
    ([2000, 1999], 256, 1000, 990, 16, 900),               # the last ones reach below the budget
    ([700], 16, 1, 1, 0, 0),
    ([700], 16, 10, 5, 5, 0),
    ([700, 33], 16, 10, 5, 0, 5),
    ([5000, 8000, 100, 4097], 16, 4096, 2048, 4, 512),
    ([40, 35], 1, 30, 20, 2, 3),                           # blocks of one token
]


@pytest.mark.parametrize("levels", [0, 2, 1], ids=["", "ties", "zeros"])
@pytest.mark.parametrize("ctx,bs,limit,budget,sinks,recent", RULES)
def test_plan(B, levels, ctx, bs, limit, budget, sinks, recent):
    p = Plan(ctx, bs, limit, budget, sinks, recent, seed=limit + bs, levels=levels)
    p.check(B)
    p.check(B, in_place=True)


def test_plan_of_special_weights(B):
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    for i, x in enumerate((np.nan, -np.nan, -1.0, -np.inf, np.inf, np.inf, -0.0, 1e-42, 0.0)):
        p.weights[p.tables[0, 2], i] = x
        p.weights[p.tables[1, 5], 3 + i] = x
    got, want = p.run(B), p.want()
    assert np.array_equal(got[0], want[0])


def test_plan_of_subnormal_weights(B):
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=4)
    p.weights = (np.arange(p.N * 16).reshape(p.N, 16) % 91).astype(np.float32) * np.float32(1e-45)
    p.check(B)


def test_plan_of_many_sequences_and_a_long_one(B):
    """More sequences than the second pass takes at once; contexts past what shared
    memory holds."""
    r = np.random.default_rng(2)
    p = Plan(r.integers(0, 80, size=2500), 16, 50, 30, 1, 5, seed=7)
    p.check(B)
    p.check(B, in_place=True)
    p = Plan([90000, 70001, 12], 16, 60000, 30000, 4, 1000, seed=8)
    p.check(B)
    p.check(B, in_place=True, max_ctx=90100)


def test_plan_refused_as_a_whole(B):
    from paged_kv_cache_96_gb300 import binding as L
    cases = []
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    cases.append((p, L.DEVERR_CONTEXT_RANGE, {}))
    p.ctx = np.array([-1, 150])
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    p.ctx = np.array([209, 150])                            # past the table
    cases.append((p, L.DEVERR_CONTEXT_RANGE, dict(max_ctx=209)))
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    cases.append((p, L.DEVERR_CONTEXT_RANGE, dict(max_ctx=199)))
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    p.count = -1
    cases.append((p, L.DEVERR_BLOCK_RANGE, {}))
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    p.count = p.N - 14                                      # 15 blocks come back
    cases.append((p, L.DEVERR_BLOCK_RANGE, {}))
    for in_place in (False, True):
        for p, flag, kw in cases:
            p.err.zero_()
            got = p.run(B, in_place, **dict(kw))
            assert int(p.err.item()) == flag
            assert (got[0] == -1).all() and np.array_equal(got[1], p.ctx)
            assert np.array_equal(got[2], p.free) and got[3] == p.count
            assert np.array_equal(got[4], p.weights) or (not in_place and (got[4] == -2).all())
    p.count = p.N - 15
    p.err.zero_()
    got = p.run(B)
    assert int(p.err.item()) == 0 and got[3] == p.N


def test_plan_with_a_bad_table_entry(B):
    from paged_kv_cache_96_gb300 import binding as L
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    want = p.want()
    for bad, j in ((-5, 1), (p.N, 1), (1 << 30, 12)):
        keep = p.tables[0, j]
        p.tables[0, j] = bad
        p.err.zero_()
        got = p.run(B)
        p.tables[0, j] = keep
        assert int(p.err.item()) == L.DEVERR_BLOCK_RANGE
        assert got[0].max() < p.N * 16 and np.array_equal(got[0][1], want[0][1])
        assert np.array_equal(got[1], want[1]) and got[3] == want[3]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.uint8])
@pytest.mark.parametrize("K,D,bs", [(8, 128, 16), (1, 64, 16), (3, 64, 32), (5, 80, 1), (40, 128, 2)])
def test_moves(B, dtype, K, D, bs):
    r = np.random.default_rng(K)
    N = 60
    g = torch.Generator().manual_seed(K)
    kc, vc = (torch.randint(0, 255, (N, bs, K, D * (1 if dtype is torch.uint8 else 2)),
                            generator=g, dtype=torch.uint8).view(dtype) for _ in range(2))
    slots = r.permutation(N * bs)
    n = min(20, N * bs // 2)
    moves = np.stack([slots[:n], slots[n:2 * n]], 1)
    listed = np.full((3, n + 11, 2), -1, dtype=np.int32)
    listed[1, 5:5 + n] = moves
    listed[2, 0] = 3, -1
    listed[0, 1] = -4, 3
    got = [x.clone().cuda() for x in (kc, vc)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.pa_move_tokens(*got, i32(listed), error_word=err)
    assert int(err.item()) == 0
    for x, y in zip(got, (kc, vc)):
        raw = y.view(torch.uint8).clone().view(N * bs, -1)
        raw[moves[:, 1]] = raw[moves[:, 0]]
        assert torch.equal(x.cpu().view(torch.uint8).view(N * bs, -1), raw)


def test_moves_flag_slots_past_the_pool(B):
    from paged_kv_cache_96_gb300 import binding as L
    kc = torch.arange(4 * 16 * 64).view(4, 16, 1, 64).to(torch.float16).cuda()
    vc = -kc
    a, b = kc.clone(), vc.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([64, 3], [3, 64], [1 << 30, 3], [3, (1 << 31) - 1]):
        err.zero_()
        B.pa_move_tokens(a, b, i32([[0, 9], bad]), error_word=err)
        assert int(err.item()) == L.DEVERR_SLOT_RANGE
        kc[0, 9], vc[0, 9] = kc[0, 0], vc[0, 0]
        assert torch.equal(a, kc) and torch.equal(b, vc)


def test_rows_past_32_bits(B):
    """Slots whose rows lie past 4 GB of a pool."""
    N, bs, K, D = 40000, 16, 32, 128
    if torch.cuda.mem_get_info()[0] < 4 * N * bs * K * D:
        pytest.skip("not enough memory")
    kc, vc = (torch.zeros((N, bs, K, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[N - 1, 15], vc[N - 1, 15] = 3.0, 4.0
    kc[N // 2, 1], vc[N // 2, 1] = 5.0, 6.0
    B.pa_move_tokens(kc, vc, i32([[N * bs - 1, 2], [N // 2 * bs + 1, N * bs - 3]]))
    assert (kc[0, 2] == 3).all() and (vc[0, 2] == 4).all()
    assert (kc[N - 1, 13] == 5).all() and (vc[N - 1, 13] == 6).all()
    assert int((kc != 0).sum()) == 4 * K * D
