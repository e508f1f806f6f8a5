"""Evictions from the same sequences again and again: the tokens that arrived last stay,
wherever earlier evictions have moved them.

Each token is known by its number of arrival, which its K row holds."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_context_step import Engine  # noqa: E402
from test_gpu_eviction import RULES, Plan, i32  # noqa: E402


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


def evict(ids, weights, total, limit, budget, sinks, recent, newest=True):
    """One sequence by the definition: the tokens at its places afterwards and the moves as
    places, from its tokens (numbers of arrival, in the order of their places) and their
    weights.  `total` have arrived in all; newest: by age, else by place."""
    c = len(ids)
    if c <= limit:
        return list(ids), []
    last = {p for p in range(sinks, c) if ids[p] >= total - recent} if newest else \
        set(range(c - recent, c))
    middle = [p for p in range(sinks, c) if p not in last]
    middle.sort(key=lambda p: (-weights[p], p))
    kept = set(range(sinks)) | last | set(middle[:budget - sinks - len(last)])
    late = [p for p in range(budget, c) if p in kept]
    holes = [p for p in range(budget) if p not in kept]
    assert len(kept) == budget and len(late) == len(holes)
    after = list(ids[:budget])
    for a, b in zip(late, holes):
        after[b] = ids[a]
    return after, list(zip(late, holes))


class Cache:
    """Sequences that grow and are evicted from; the host's side keeps lists of tokens."""

    def __init__(self, S, bs, most, aged, seed=0):
        self.r = np.random.default_rng(seed)
        MB = -(-most // bs)
        N = S * MB + 3
        self.S, self.bs, self.N, self.most, self.aged = S, bs, N, most, aged
        self.tables = np.full((S, MB), -3, dtype=np.int32)
        self.free, self.count = self.r.permutation(N).astype(np.int32), N
        self.ids, self.total = [[] for _ in range(S)], [0] * S
        self.kc = torch.zeros((N, bs, 1, 8), dtype=torch.float16, device="cuda")
        self.vc = self.kc.clone()
        self.ages = torch.full((N, bs), -999, dtype=torch.int32, device="cuda")
        self.numbered, self.gone = i32(np.zeros(S)), i32(np.zeros(S))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def slots(self, s, places):
        p = np.asarray(places, dtype=int)
        return self.tables[s, p // self.bs].astype(int) * self.bs + p % self.bs

    def rows(self):
        """Token that each slot's K row holds (V: its negative), as exact fp16 digits."""
        k, v = (x.view(self.N * self.bs, 8)[:, :2].float().cpu().numpy() for x in (self.kc, self.vc))
        assert np.array_equal(k, -v)
        return (k[:, 0] * 1024 + k[:, 1]).astype(int)

    def grow(self, s, n):
        have, c = -(-len(self.ids[s]) // self.bs), len(self.ids[s])
        for j in range(have, -(-(c + n) // self.bs)):
            self.count -= 1
            self.tables[s, j] = self.free[self.count]
        new = np.arange(self.total[s], self.total[s] + n)
        self.ids[s] += new.tolist()
        self.total[s] += n
        at = torch.as_tensor(self.slots(s, np.arange(c, c + n))).cuda()
        digits = torch.as_tensor(np.stack([new // 1024, new % 1024], 1)).to(torch.float16).cuda()
        self.kc.view(-1, 8)[at, :2] = digits
        self.vc.view(-1, 8)[at, :2] = -digits

    def step(self, B, rule, in_place, all_newest=True):
        limit, budget, sinks, recent = rule
        ctx = [len(x) for x in self.ids]
        # older tokens have more, and what no token holds is worth most
        weights = np.full((self.N, self.bs), 1e9, dtype=np.float32)
        w = []
        for s, c in enumerate(ctx):
            x = self.r.random(c) * (1 + self.total[s] - np.asarray(self.ids[s], dtype=float))
            x = np.round(x * 4) / 4               # some are equal
            w.append(x)
            weights.flat[self.slots(s, np.arange(c))] = x
        dev_w, dev_ctx, count = torch.as_tensor(weights).cuda(), i32(ctx), i32([self.count])
        w_out = dev_w if in_place else torch.full_like(dev_w, -2)
        ctx_out = dev_ctx if in_place else dev_ctx.clone().fill_(-2)
        count_out = count if in_place else i32([-2])
        M = max(1, min(budget, self.most - budget))
        moves = torch.full((self.S, M, 2), 55, dtype=torch.int32, device="cuda")
        free, tables = i32(self.free), i32(self.tables)
        more = dict(arrivals=self.ages, numbered_lens=self.numbered, evicted=self.gone) \
            if self.aged else {}
        B.pa_plan_eviction(moves, ctx_out, count_out, w_out, tables, dev_ctx, dev_w, free, count,
                           self.most, *rule, error_word=self.err, **more)
        B.pa_move_tokens(self.kc, self.vc, moves, error_word=self.err)
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        want_moves = np.full((self.S, M, 2), -1)
        cut = 0
        for s, c in enumerate(ctx):
            after, places = evict(self.ids[s], w[s], self.total[s], *rule, newest=self.aged)
            for i, (a, b) in enumerate(places):
                want_moves[s, i] = self.slots(s, [a, b])
            if c > limit:
                cut += 1
                # what this is about
                newest = set(range(self.total[s] - recent, self.total[s]))
                assert newest & set(self.ids[s]) <= set(after)
                assert not all_newest or newest <= set(after)
            for j in range(-(-len(after) // self.bs), -(-c // self.bs)):
                self.free[self.count] = self.tables[s, j]
                self.count += 1
            weight_of = dict(zip(self.ids[s], w[s]))
            self.ids[s] = after
            at = self.slots(s, np.arange(len(after)))
            assert np.array_equal(self.rows()[at], after)
            got = w_out.cpu().numpy().flat[at]
            assert np.array_equal(got, np.array([weight_of[i] for i in after], dtype=np.float32))
            if self.aged and c > limit:
                assert np.array_equal(self.ages.cpu().numpy().flat[at], after)
        assert np.array_equal(moves.cpu().numpy(), want_moves)
        assert ctx_out.tolist() == [len(x) for x in self.ids]
        assert int(count_out.item()) == self.count
        assert np.array_equal(free.cpu().numpy()[:self.count], self.free[:self.count])
        if self.aged:
            assert self.gone.tolist() == [t - len(x) for t, x in zip(self.total, self.ids)]
        return cut


AGED = [
    # limit, budget, sinks, recent, block, tokens a step
    (64, 64, 4, 16, 16, 1),
    (64, 64, 1, 63, 16, 1),                    # nothing is chosen by weight
    (40, 40, 0, 40, 1, 3),                     # the last 40 alone, blocks of one token
    (70, 64, 4, 32, 64, 2),
    (72, 64, 60, 3, 16, 1),
    (100, 33, 2, 5, 16, 30),
    (64, 64, 4, 0, 16, 1),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("limit,budget,sinks,recent,bs,new", AGED)
def test_the_newest_tokens_survive_every_eviction(B, in_place, limit, budget, sinks, recent, bs,
                                                  new):
    c = Cache(3, bs, limit + 3 * new + 8, True, seed=limit + recent)
    cuts = 0
    for k in range(60):
        for s in range(3):
            c.grow(s, [new, k % (new + 1), 2 * new][s])
        cuts += c.step(B, (limit, budget, sinks, recent), in_place)
    assert cuts >= 5


def test_rules_that_change_between_evictions(B):
    """A smaller budget, fewer first tokens, more last ones: of these, those that are still
    cached."""
    c = Cache(2, 16, 300, True, seed=5)
    rules = [(200, 150, 4, 10), (120, 110, 4, 70), (110, 110, 4, 30), (90, 60, 2, 10),
             (60, 60, 9, 20)]
    for k in range(40):
        for s in range(2):
            c.grow(s, 17 - 5 * s)
        c.step(B, rules[min(k // 8, 4)], k % 2 == 0, all_newest=False)


@pytest.mark.parametrize("max_ctx", [60000, 50000])
def test_long_contexts(B, max_ctx):
    """Longer than the plan's shared memory holds, and as long as it does."""
    c = Cache(2, 16, max_ctx, True, seed=7)
    c.grow(0, max_ctx - 4000)
    c.grow(1, max_ctx - 20000)
    rule = (max_ctx - 3000, max_ctx - 3001, 4, 1000)
    for k in range(4):
        c.grow(0, 1500 + k)
        c.grow(1, 9000 if k < 2 else 300)
        c.step(B, rule, k % 2 == 0)
    assert c.gone.min() > 0


@pytest.mark.parametrize("limit,budget,sinks,recent,new", [(79, 64, 4, 16, 1), (80, 64, 0, 17, 3),
                                                           (40, 40, 3, 1, 1)])
def test_by_place_where_enough_tokens_come_between(B, limit, budget, sinks, recent, new):
    """limit - budget + 1 >= num_recent: the last places hold the newest tokens."""
    c = Cache(3, 16, limit + 2 * new + 8, False, seed=limit)
    for k in range(70):
        for s in range(3):
            c.grow(s, new if s else 1)
        c.step(B, (limit, budget, sinks, recent), k % 2 == 0)


@pytest.mark.parametrize("levels", [0, 2], ids=["", "ties"])
@pytest.mark.parametrize("ctx,bs,limit,budget,sinks,recent", RULES)
def test_a_first_eviction_is_that_by_place(B, levels, ctx, bs, limit, budget, sinks, recent):
    for in_place in (False, True):
        p = Plan(ctx, bs, limit, budget, sinks, recent, seed=limit + bs, levels=levels)
        ages = torch.full((p.N, bs), 1 << 30, dtype=torch.int32, device="cuda")
        numbered, gone = i32(np.zeros(len(ctx))), i32(np.full(len(ctx), (1 << 31) - 20))
        p.check(B, in_place, arrivals=ages, numbered_lens=numbered, evicted=gone)
        over = np.asarray(ctx) > limit
        assert numbered.tolist() == np.where(over, budget, 0).tolist()
        lost = (gone.cpu().numpy().astype(np.int64) - ((1 << 31) - 20)) % (1 << 32)
        assert lost.tolist() == np.where(over, np.asarray(ctx) - budget, 0).tolist()


def ages_of(p, seed=1):
    """Numbers of arrival for all but the last 30 tokens of each context, out of order."""
    r = np.random.default_rng(seed)
    ages = np.full((p.N, p.bs), -5, dtype=np.int32)
    numbered = np.maximum(p.ctx - 30, 0)
    for s, n in enumerate(numbered):
        places = np.arange(n)
        ages[p.tables[s, places // p.bs], places % p.bs] = r.permutation(n + 40)[:n]
    return i32(ages), i32(numbered), i32([40] * len(p.ctx))


def test_a_refused_plan_leaves_ages_as_they_were(B):
    from paged_kv_cache_96_gb300 import binding as L
    for in_place in (False, True):
        for why in ("length", "stack"):
            p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
            state = ages_of(p)
            if why == "length":
                p.ctx = np.array([200, -1])
            else:
                p.count = p.N
            before = [x.clone() for x in state]
            got = p.run(B, in_place, arrivals=state[0], numbered_lens=state[1], evicted=state[2])
            assert int(p.err.item()) == (L.DEVERR_CONTEXT_RANGE if why == "length" else
                                         L.DEVERR_BLOCK_RANGE)
            assert (got[0] == -1).all()
            assert all(torch.equal(a, b) for a, b in zip(before, state))


def test_a_numbered_length_outside_its_context_counts_as_none(B):
    from paged_kv_cache_96_gb300 import binding as L
    for bad in (201, -1, 1 << 30, -(1 << 31)):
        p = Plan([200, 150, 50], 16, 100, 60, 2, 8, seed=3)
        ages, numbered, gone = ages_of(p)
        numbered[0] = numbered[1] = bad
        got = p.run(B, arrivals=ages, numbered_lens=numbered, evicted=gone)
        assert int(p.err.item()) == L.DEVERR_CONTEXT_RANGE
        want = p.want()                        # as if nothing had been evicted before
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert numbered.tolist() == [60, 60, 20] and gone.tolist() == [180, 130, 40]


def test_a_bad_table_entry_and_ages(B):
    from paged_kv_cache_96_gb300 import binding as L
    for bad, j in ((-5, 1), (1 << 20, 12)):
        p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
        ages, numbered, gone = ages_of(p)
        want = p.run(B, arrivals=ages.clone(), numbered_lens=numbered.clone(), evicted=gone.clone())
        p.tables[0, j] = bad
        got = p.run(B, arrivals=ages, numbered_lens=numbered, evicted=gone)
        assert int(p.err.item()) == L.DEVERR_BLOCK_RANGE
        assert got[0].max() < p.N * 16 and np.array_equal(got[0][1], want[0][1])
        assert np.array_equal(got[1], want[1]) and numbered.tolist() == [60, 60]


def test_ages_come_together_and_in_shape(B):
    p = Plan([200, 150], 16, 100, 60, 2, 8, seed=3)
    ages, numbered, gone = ages_of(p)
    good = dict(arrivals=ages, numbered_lens=numbered, evicted=gone)
    for bad in (dict(arrivals=None), dict(numbered_lens=None), dict(evicted=None),
                dict(arrivals=ages[:-1]), dict(arrivals=ages.view(-1)), dict(arrivals=ages.float()),
                dict(arrivals=ages.t()), dict(arrivals=ages.cpu()), dict(numbered_lens=numbered[:1]),
                dict(numbered_lens=numbered.long()), dict(evicted=torch.cat([gone, gone])),
                dict(evicted=gone.cpu()), dict(arrivals=5)):
        with pytest.raises((TypeError, ValueError)):
            p.run(B, **dict(good, **bad))
    assert int(p.err.item()) == 0


class Aged(Engine):
    """Decode steps whose sequences are evicted from as soon as they pass their budget."""

    LIMIT, BUDGET, SINKS, RECENT = 90, 90, 3, 25

    def __init__(self, *args):
        super().__init__(*args)
        self.ages = torch.full((self.N, self.BS), -7, dtype=torch.int32, device="cuda")
        self.numbered = torch.zeros_like(self.gone)

    def evict(self):
        B = self.B
        B.pa_plan_eviction(self.moves, self.ctx, self.count, self.weights, self.tables, self.ctx,
                           self.weights, self.free, self.count, self.max_ctx, self.LIMIT,
                           self.BUDGET, self.SINKS, self.RECENT, error_word=self.err,
                           arrivals=self.ages, numbered_lens=self.numbered, evicted=self.gone)
        self.weighted.copy_(self.ctx)
        B.pa_move_tokens(self.kc, self.vc, self.moves, error_word=self.err)
        B.pa_summarize_blocks(self.codes, self.scales, self.kc, self.tables, self.ctx,
                              error_word=self.err)

    def decode(self):
        self.weights_step()
        self.evict()


def test_a_step_that_evicts_every_time(B):
    """Prompts, then decode steps as one replayed graph each: weights added up, an eviction a
    sequence and step, and the newest tokens' values still in the cache."""
    e = Aged(B, torch.bfloat16, False, 8, 2, 64)
    graphs = {}
    queue = torch.cuda.Stream()
    with torch.cuda.stream(queue):
        for name in ("sparse_step", "decode"):
            getattr(e, name)()                 # nobody has a token yet
        torch.cuda.synchronize()
        for name in ("sparse_step", "decode"):
            graphs[name] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[name], stream=queue):
                getattr(e, name)()
    torch.cuda.synchronize()
    values = [[] for _ in range(e.S)]          # V rows of each sequence's tokens
    for k in range(70):
        new = [30, 20, 0, 45] if k < 2 else [1, 1, 1, 1]
        e.new.copy_(torch.as_tensor(new))
        e.qkv.copy_(torch.randn(e.qkv.shape, generator=torch.Generator().manual_seed(k)))
        at = 0
        for s, n in enumerate(new):
            values[s] += list(e.qkv[at:at + n, -e.K:].cpu())
            at += n
        graphs["sparse_step" if k < 2 else "decode"].replay()
        torch.cuda.synchronize()
        assert int(e.err.item()) == 0
        tables, ctx, gone, ages, numbered = e.host("tables", "ctx", "gone", "ages", "numbered")
        for s, c in enumerate(ctx):
            total = len(values[s])
            assert c == (min(total, e.BUDGET) if k >= 2 else total) and gone[s] == total - c
            p = np.arange(c)
            ids = ages[tables[s][p // e.BS], p % e.BS] if gone[s] else p
            assert numbered[s] == (e.BUDGET if gone[s] else 0)
            assert len(set(ids.tolist())) == c
            assert set(range(total - min(total, e.RECENT), total)) <= set(ids.tolist())
            assert ids[:e.SINKS].tolist() == list(range(min(c, e.SINKS)))
            if c:
                got = e.vc[torch.as_tensor(tables[s][p // e.BS]).long(), torch.as_tensor(p % e.BS)]
                assert torch.equal(got.cpu(), torch.stack([values[s][i] for i in ids]))
    assert (gone[[0, 1, 3]] > 0).all()
