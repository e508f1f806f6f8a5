"""pa_build_step_maps against the definition taken one block and one token at a
time: every output integer equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import operator_refs as R  # noqa: E402


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


class Maps:
    """Inputs and outputs of one call on the device."""

    def __init__(self, tables, ctx, new, free, count, bs, capacity):
        t = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        f = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bs, self.N = bs, len(free)
        self.tables, self.ctx, self.new, self.free, self.count = \
            t(tables), t(ctx), t(new), t(free), t([count])
        S = len(ctx)
        self.start, self.seq, self.pos, self.slot = f(S + 1), f(capacity), f(capacity), f(capacity)
        self.ctx_out, self.count_out, self.err = f(S), f(1), torch.zeros(1, dtype=torch.int32,
                                                                         device="cuda")

    def call(self, B, in_place=False, stream=None):
        if in_place:
            self.ctx_out, self.count_out = self.ctx, self.count
        B.pa_build_step_maps(self.tables, self.ctx, self.new, self.free, self.count, self.bs,
                             self.N, self.start, self.seq, self.pos, self.slot, self.ctx_out,
                             self.count_out, error_word=self.err, stream=stream)

    def got(self):
        torch.cuda.synchronize()
        c = lambda x: x.cpu().numpy()  # noqa: E731
        return dict(start=c(self.start), seq=c(self.seq), pos=c(self.pos), slot=c(self.slot),
                    ctx=c(self.ctx_out), tables=c(self.tables), free=c(self.free),
                    count=int(self.count_out.item()))


def check(got, want):
    for k in ("start", "seq", "pos", "slot", "ctx", "tables", "free"):
        assert np.array_equal(got[k], want[k]), k
    assert got["count"] == want["count"]


def make(rng, S, bs, MB, longest, spare=40, finished=0.2, idle=0.1, one=0.5):
    cap = MB * bs
    new = rng.integers(1, longest + 1, size=S)
    new[rng.random(S) < one] = 1
    new[rng.random(S) < idle] = 0
    ctx = rng.integers(0, np.maximum(1, cap - new + 1))
    new[rng.random(S) < finished] = -1
    have = -(-ctx // bs)
    need = int((-(-(ctx + np.maximum(new, 0)) // bs) - have)[new >= 0].sum())
    ids = rng.permutation(int(have.sum()) + need + spare).astype(np.int32)
    tables = np.full((S, MB), -7, dtype=np.int32)  # entries past a sequence's own: never read
    at = 0
    for s in range(S):
        tables[s, :have[s]] = ids[at:at + have[s]]
        at += have[s]
    free = np.full(len(ids), -5, dtype=np.int32)
    free[:len(ids) - at] = ids[at:]
    return tables, ctx, new, free, len(ids) - at


@pytest.mark.parametrize("S,bs,MB,longest,pad", [
    (1, 16, 4, 1, 0), (1, 16, 40, 600, 0), (2, 16, 8, 100, 5), (4, 1, 60, 40, 1),
    (31, 16, 20, 1, 0), (33, 24, 20, 17, 3), (61, 16, 64, 512, 100), (128, 16, 64, 1, 0),
    (1000, 32, 8, 9, 31), (1023, 16, 16, 2, 0), (1025, 16, 16, 2, 0), (3000, 16, 12, 30, 7),
    (9001, 7, 10, 3, 64), (20000, 16, 2, 2, 0)])
def test_matches_the_definition(B, S, bs, MB, longest, pad):
    rng = np.random.default_rng(S * 131 + bs)
    for finished, idle, one in ((0.2, 0.1, 0.5), (0.0, 0.0, 1.0), (0.9, 0.05, 0.0)):
        tables, ctx, new, free, count = make(rng, S, bs, MB, longest, finished=finished,
                                             idle=idle, one=one)
        T = int(np.maximum(new, 0).sum()) + pad
        want = R.step_maps(tables, ctx, new, free, count, bs, T)
        assert want is not None
        m = Maps(tables, ctx, new, free, count, bs, T)
        m.call(B)
        check(m.got(), want)
        assert int(m.err.item()) == 0


def test_one_long_prompt_among_many(B):
    """A prompt of 60,000 tokens between requests of one: tokens and blocks are
    shared out whatever the lengths."""
    S, bs, MB = 65, 16, 4000
    new = np.ones(S, dtype=np.int64)
    new[40] = 60000
    ctx = np.arange(S) * 3
    ctx[40] = 0
    have = -(-ctx // bs)
    rng = np.random.default_rng(5)
    ids = rng.permutation(int(have.sum()) + 3900).astype(np.int32)
    tables = np.zeros((S, MB), dtype=np.int32)
    at = 0
    for s in range(S):
        tables[s, :have[s]] = ids[at:at + have[s]]
        at += have[s]
    free = np.zeros(len(ids), dtype=np.int32)
    free[:len(ids) - at] = ids[at:]
    T = int(new.sum())
    want = R.step_maps(tables, ctx, new, free, len(ids) - at, bs, T)
    m = Maps(tables, ctx, new, free, len(ids) - at, bs, T)
    m.call(B)
    check(m.got(), want)


def test_nothing_to_do(B):
    """No sequences, or none with a token: offsets 0, the token arrays padding."""
    for S, T in ((0, 0), (0, 5), (3, 0), (3, 4)):
        tables = np.zeros((S, 4), dtype=np.int32)
        tables[:, 0] = np.arange(S)
        free = np.arange(10, dtype=np.int32)
        m = Maps(tables, np.full(S, 5), np.zeros(S), free, 4, 16, T)
        m.call(B)
        check(m.got(), R.step_maps(tables, np.full(S, 5), np.zeros(S, dtype=int), free, 4, 16, T))
        assert int(m.err.item()) == 0


BASE = dict(ctx=[20, 0, 16], new=[3, 17, -1], count=6, capacity=24)
REFUSED = [
    (dict(ctx=[-1, 0, 16]), "DEVERR_CONTEXT_RANGE"),
    (dict(new=[-2, 17, -1]), "DEVERR_CONTEXT_RANGE"),
    (dict(ctx=[65, 0, 16]), "DEVERR_CONTEXT_RANGE"),
    (dict(new=[45, 0, -1], capacity=64), "DEVERR_CONTEXT_RANGE"),   # 20 + 45 > 4 * 16
    (dict(new=[2 ** 31 - 1, 0, -1]), "DEVERR_CONTEXT_RANGE"),
    (dict(capacity=19), "DEVERR_TOKEN_RANGE"),
    (dict(count=-1), "DEVERR_BLOCK_RANGE"),
    (dict(count=12), "DEVERR_BLOCK_RANGE"),                         # 12 + 1 given back > 12
    (dict(count=0, new=[13, 17, 0], capacity=40), "DEVERR_OUT_OF_BLOCKS"),
]


@pytest.mark.parametrize("change,flag", REFUSED, ids=[f"{c}" for c, _ in REFUSED])
@pytest.mark.parametrize("in_place", [False, True])
def test_refused_steps_change_nothing(B, change, flag, in_place):
    a = dict(BASE, **change)
    tables = np.arange(12, dtype=np.int32).reshape(3, 4)
    free = np.arange(12, dtype=np.int32)[::-1].copy()
    assert R.step_maps(tables, a["ctx"], a["new"], free, a["count"], 16, a["capacity"]) is None
    m = Maps(tables, a["ctx"], a["new"], free, a["count"], 16, a["capacity"])
    m.call(B, in_place)
    got = m.got()
    assert int(m.err.item()) == getattr(B, flag)
    assert np.array_equal(got["tables"], tables) and np.array_equal(got["free"], free)
    assert list(got["ctx"]) == a["ctx"] and got["count"] == a["count"]
    assert (got["start"] == 0).all()
    for k in ("seq", "pos", "slot"):
        assert (got[k] == -1).all()


def test_base_of_the_refusals_is_taken(B):
    tables = np.arange(12, dtype=np.int32).reshape(3, 4)
    free = np.arange(12, dtype=np.int32)[::-1].copy()
    want = R.step_maps(tables, BASE["ctx"], BASE["new"], free, 6, 16, 24)
    m = Maps(tables, BASE["ctx"], BASE["new"], free, 6, 16, 24)
    m.call(B, in_place=True)
    check(m.got(), want)


def test_bad_blocks_are_flagged_and_give_no_slot(B):
    """A stack entry outside the pool leaves -1 in the table, a bad table entry
    is not used; the other sequences get theirs."""
    tables = np.array([[3, 0], [99, 0], [-4, 0]], dtype=np.int32)
    free = np.array([5, 50, 6, 0], dtype=np.int32)  # pops 6, then 50
    m = Maps(tables, [16, 4, 4], [2, 13, 1], free, 3, 16, 20)
    m.call(B)
    got = m.got()
    assert int(m.err.item()) == B.DEVERR_BLOCK_RANGE
    assert got["tables"][0, 1] == -1 and got["tables"][1, 1] == -1  # 6 and 50 of a pool of 4
    assert (got["slot"] == -1).all() and list(got["start"]) == [0, 2, 15, 16]
    # the same with blocks inside the pool
    free = np.array([1, 2, 0, 0], dtype=np.int32)
    tables = np.array([[3, 0], [99, 0]], dtype=np.int32)
    m = Maps(tables, [16, 4], [2, 13], free, 3, 16, 15)
    m.call(B)
    got = m.got()
    assert list(got["slot"][:2]) == [0, 1] and got["slot"][14] == 2 * 16
    assert (got["slot"][2:14] == -1).all()
    assert int(m.err.item()) == B.DEVERR_BLOCK_RANGE


@pytest.mark.parametrize("S,MB", [(37, 30), (1500, 10)])
def test_captured_step_walks_its_own_state(B, S, MB):
    """In place: a captured graph replayed twenty times is twenty steps; finished
    requests' blocks come back to others."""
    rng = np.random.default_rng(S)
    tables, ctx, new, free, count = make(rng, S, 16, MB, 3, spare=S * MB, finished=0.0)
    ctx = np.minimum(ctx, (MB - 6) * 16)
    T = 3 * S
    m = Maps(tables, ctx, new, free, count, 16, T)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.call(B, in_place=True)  # one step ahead of the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.call(B, in_place=True)
    state = dict(tables=tables, free=free, ctx=ctx, count=count)
    for i in range(21):
        nw = new.copy()
        if i == 7:
            nw[::3] = -1
        if i:
            m.new.copy_(torch.as_tensor(nw.astype(np.int32)))
            g.replay()
        want = R.step_maps(state["tables"], state["ctx"], nw, state["free"], state["count"], 16, T)
        check(m.got(), want)
        state = want
    assert int(m.err.item()) == 0


def test_binding_checks_every_tensor(B):
    rng = np.random.default_rng(5)
    tables, ctx, new, free, count = make(rng, 6, 16, 8, 20, finished=0.0)
    m = Maps(tables, ctx, new, free, count, 16, 90)
    for name in ("tables", "ctx", "new", "free", "count", "start", "seq", "pos", "slot", "ctx_out",
                 "count_out", "err"):
        good = getattr(m, name)
        for bad, error in ((good.long(), TypeError), (good.cpu(), ValueError), (None, TypeError),
                           (good.repeat_interleave(2, -1)[..., ::2], ValueError)):
            if name == "err" and bad is None or good.numel() == 1 and bad is not None and \
                    bad.is_cuda and bad.dtype == good.dtype:
                continue                    # (no error word is fine; one entry is dense)
            setattr(m, name, bad)
            with pytest.raises(error):
                m.call(B)
            setattr(m, name, good)
    for name in ("ctx", "new", "start", "pos", "slot", "ctx_out"):
        good = getattr(m, name)
        setattr(m, name, good[1:])
        with pytest.raises(ValueError):
            m.call(B)
        setattr(m, name, good)
    torch.cuda.synchronize()
    assert bool((m.seq == 77).all()) and np.array_equal(m.tables.cpu().numpy(), tables)
    m.call(B)
    check(m.got(), R.step_maps(tables, ctx, new, free, count, 16, 90))
