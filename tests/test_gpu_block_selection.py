"""Block bounds and block selection against their definitions, for equality.

Pools hold NaN wherever no token below the context is, and table entries past the
context point outside the pool."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import context_refs as C  # noqa: E402

KINDS = {"bf16": (torch.bfloat16, False), "f16": (torch.float16, False),
         "fp8": (torch.bfloat16, True)}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Keys:
    """A key pool of shuffled blocks for contexts `ctx`."""

    def __init__(self, ctx, K, D, bs, kind, seed=0, amp=1.0, spare=3):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.bs = np.asarray(ctx), bs
        blocks = -(-self.ctx // bs)
        self.N, MB = int(blocks.sum()) + spare, max(1, int(blocks.max()))
        ids = r.permutation(self.N)
        self.tables = np.full((len(ctx), MB), self.N + 7, dtype=np.int32)
        live = np.zeros((self.N, bs), dtype=bool)
        at = 0
        for s, n in enumerate(blocks):
            self.tables[s, :n] = ids[at:at + n]
            at += n
            p = np.arange(self.ctx[s])
            live[self.tables[s, p // bs], p % bs] = True
        dtype, fp8 = KINDS[kind]
        x = torch.randn((self.N, bs, K, D), generator=g) * amp
        hide = torch.as_tensor(~live)[..., None, None].expand(x.shape)
        if fp8:
            x = (x * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            x = x.masked_fill(hide, 0x7F)
        else:
            x = x.to(dtype).masked_fill(hide, float("nan"))
        self.keys = x
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def summarize(self, B, start=None, tables=None, ctx=None, fill=77):
        N, _, K, D = self.keys.shape
        codes = torch.full((N, K, 2, D), fill, dtype=torch.int8, device="cuda")
        scales = torch.full((N, K), float(fill), device="cuda")
        B.pa_summarize_blocks(codes, scales, self.keys.cuda(),
                              i32(self.tables if tables is None else tables),
                              i32(self.ctx if ctx is None else ctx),
                              query_start=None if start is None else i32(start),
                              error_word=self.err)
        torch.cuda.synchronize()
        return codes.cpu().numpy(), scales.cpu().numpy()

    def want(self, start=None, fill=77, tables=None):
        N, _, K, D = self.keys.shape
        codes = np.full((N, K, 2, D), fill, dtype=np.int8)
        scales = np.full((N, K), float(fill), dtype=np.float32)
        C.summarize(codes, scales, C.values(self.keys),
                    self.tables if tables is None else tables, self.ctx, start)
        return codes, scales


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("K,D,bs,ctx", [
    (1, 64, 16, [1]), (4, 64, 16, [1, 15, 16, 17, 500]), (3, 128, 16, [0, 33, 0, 64, 47]),
    (8, 128, 32, [31, 32, 33, 200]), (2, 128, 256, [1, 255, 257, 513]), (5, 64, 64, [64, 129]),
    (2, 64, 128, [127, 128, 300]),
])
def test_bounds_of_whole_contexts(B, kind, K, D, bs, ctx):
    k = Keys(ctx, K, D, bs, kind, seed=K * D + bs)
    got, want = k.summarize(B), k.want()
    assert int(k.err.item()) == 0
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])


@pytest.mark.parametrize("kind", list(KINDS))
def test_bounds_of_the_steps_blocks_alone(B, kind):
    ctx = [1, 16, 17, 40, 100, 33, 0, 64]
    new = [1, 1, 1, 0, 37, 33, 0, 48]
    k = Keys(ctx, 4, 128, 16, kind, seed=3)
    start = np.concatenate([[0], np.cumsum(new)])
    got, want = k.summarize(B, start), k.want(start)
    assert int(k.err.item()) == 0
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
    assert (want[0] == 77).all(-1).any()       # some blocks were left as they were


def test_bounds_of_many_sequences(B):
    """More sequences than a CTA numbers at once, decode rows among long ones."""
    r = np.random.default_rng(5)
    ctx = r.integers(0, 60, size=1337)
    new = np.minimum(ctx, r.integers(0, 3, size=1337))
    ctx[700] = new[700] = 900
    k = Keys(ctx, 1, 64, 16, "f16", seed=6)
    start = np.concatenate([[0], np.cumsum(new)])
    got, want = k.summarize(B, start), k.want(start)
    assert int(k.err.item()) == 0
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_bounds_of_special_keys(B, kind):
    k = Keys([80, 16], 2, 64, 16, kind, seed=9)
    t = k.tables
    x = k.keys
    x[t[0, 0], 3, 0, 5] = float("nan")
    x[t[0, 1], 0, 1, 63] = float("inf")
    x[t[0, 2], 15, 0, 0] = -float("inf")
    x[t[0, 3]] = 0.0
    x[t[0, 3], 2, 1] = -0.0
    x[t[0, 4], :, 0] = torch.finfo(x.dtype).smallest_normal    # bf16: far below 2^-40
    x[t[0, 4], :, 1] = torch.finfo(x.dtype).max
    x[t[1, 0], :, 0] = 2.0 ** -14
    x[t[1, 0], 7, 0, 7] = torch.finfo(x.dtype).tiny / 4        # a subnormal beside them
    got, want = k.summarize(B), k.want()
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
    assert np.isinf(want[1]).sum() == 3 and (want[1] == 0).sum() >= 2


def test_bounds_flag_what_is_out_of_range(B):
    from paged_kv_cache_96_gb300.binding import DEVERR_BLOCK_RANGE, DEVERR_CONTEXT_RANGE
    k = Keys([40, 50], 2, 64, 16, "f16", seed=11)
    bad = k.tables.copy()
    bad[0, 1], bad[1, 0] = -1, k.N
    got = k.summarize(B, tables=bad)
    assert int(k.err.item()) == DEVERR_BLOCK_RANGE
    codes, scales = k.want()
    for s, j in ((0, 1), (1, 0)):              # skipped: as they were
        codes[k.tables[s, j]], scales[k.tables[s, j]] = 77, 77
    assert np.array_equal(got[1], scales) and np.array_equal(got[0], codes)
    for ctx, start in (([-3, 50], None), ([40, 1 << 30], None), ([40, 50], [0, 41, 50]),
                       ([40, 50], [0, -2, 50])):
        k.err.zero_()
        k.summarize(B, start=start, ctx=ctx, tables=np.clip(k.tables, 0, k.N - 1))
        assert int(k.err.item()) == DEVERR_CONTEXT_RANGE


# ---- selection ---------------------------------------------------------------------


class Bounds:
    """Coded bounds of N blocks and the tables of contexts over them."""

    def __init__(self, ctx, K, D, bs, seed=0, ties=False):
        r = np.random.default_rng(seed)
        self.ctx, self.bs = np.asarray(ctx), bs
        blocks = -(-self.ctx // bs)
        self.N, MB = int(blocks.sum()) + 2, max(1, int(blocks.max()))
        ids = r.permutation(self.N)
        self.tables = np.full((len(ctx), MB), -9, dtype=np.int32)
        at = 0
        for s, n in enumerate(blocks):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        top = 3 if ties else 128
        a, b = (r.integers(1 - top, top, size=(self.N, K, D)) for _ in range(2))
        if ties:                               # few scores: many are equal
            a[..., 4:] = b[..., 4:] = 0
        self.codes = np.stack([np.minimum(a, b), np.maximum(a, b)], 2).astype(np.int8)
        self.scales = (np.full((self.N, K), 0.25) if ties else
                       np.exp(r.normal(-4, 0.3, size=(self.N, K)))).astype(np.float32)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def select(self, B, q, seq, pos, top_k, first, last, max_ctx=None, tables=None, **kw):
        K = self.codes.shape[1]
        out = torch.full((len(seq), K, top_k), 99, dtype=torch.int32, device="cuda")
        B.pa_select_blocks(out, q.cuda(), torch.as_tensor(self.codes).cuda(),
                           torch.as_tensor(self.scales).cuda(),
                           i32(self.tables if tables is None else tables), i32(seq), i32(pos),
                           int(max(pos) + 1 if max_ctx is None else max_ctx), self.bs,
                           num_first=first, num_last=last, error_word=self.err, **kw)
        torch.cuda.synchronize()
        return out.cpu().numpy()

    def check(self, B, q, seq, pos, top_k, first, last, **kw):
        got = self.select(B, q, seq, pos, top_k, first, last, **kw)
        assert int(self.err.item()) == 0
        want = C.select(q.float().numpy(), self.codes, self.scales, self.tables, seq, pos,
                        self.bs, top_k, first, last, self.codes.shape[1])
        assert np.array_equal(got, want)
        return got


def query(T, H, D, dtype, seed=1):
    return torch.randn((T, H, D), generator=torch.Generator().manual_seed(seed)).to(dtype)


SELECT = [
    # H, K, D, bs, contexts, top_k, first, last
    (4, 4, 64, 16, [1, 16, 17, 500], 8, 1, 1),
    (8, 1, 128, 16, [300, 1000], 5, 0, 1),
    (16, 1, 64, 32, [33, 2000], 16, 2, 3),
    (10, 2, 128, 16, [900, 20, 3000], 7, 1, 2),
    (3, 1, 128, 64, [5000], 3, 1, 2),                       # nothing but first and last
    (64, 8, 128, 16, [700, 64, 65], 4, 0, 0),
    (9, 1, 64, 256, [256, 257, 9000], 1, 0, 1),
    (5, 5, 128, 16, [1030], 64, 1, 1),                      # 65 blocks of which 64
    (24, 2, 64, 16, [40000, 17, 12345], 100, 1, 4),         # clusters of several CTAs
    (2, 1, 128, 16, [100000], 129, 3, 0),
    (4, 2, 64, 16, [90000, 5000], 4, 2, 2),                 # the same in clusters
    (16, 1, 128, 16, [60000, 300], 1500, 10, 20),           # lists longer than a CTA's share
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("ties", [False, True], ids=["", "ties"])
@pytest.mark.parametrize("H,K,D,bs,ctx,top_k,first,last", SELECT)
def test_selection(B, dtype, ties, H, K, D, bs, ctx, top_k, first, last):
    x = Bounds(ctx, K, D, bs, seed=H + D + bs, ties=ties)
    seq = np.arange(len(ctx))
    x.check(B, query(len(ctx), H, D, dtype), seq, x.ctx - 1, top_k, first, last)


def test_rows_of_one_sequence_and_padding(B):
    """Several rows of a sequence at their own positions, in any order, and padding."""
    x = Bounds([1500, 400], 2, 128, 16, seed=4)
    seq = np.array([0, 0, -1, 1, 0, 1, -1, -5])
    pos = np.array([1499, 1498, -1, 399, 0, 129, 7, 20])
    got = x.check(B, query(8, 8, 128, torch.bfloat16), seq, pos, 9, 1, 1)
    assert (got[[2, 6, 7]] == -1).all() and (got[4, :, 1:] == -1).all()


def test_selection_of_special_queries_and_bounds(B):
    x = Bounds([2000], 2, 64, 16, seed=8)
    q = query(6, 8, 64, torch.bfloat16)
    q[0, 0, 3] = float("nan")                  # one head of four without a say
    q[1, :4, 0] = float("inf")                 # a group without one: the lowest blocks
    q[2] = 0
    q[3] *= 2.0 ** -50                         # below the least amplitude
    q[4] *= 2.0 ** 120
    t = x.tables[0]
    x.scales[t[50]] = x.scales[t[20]] = np.inf  # first of all, whatever the query
    x.scales[t[70]] = 0
    x.codes[t[70]] = 0
    seq, pos = np.zeros(6, dtype=int), np.full(6, 1999)
    got = x.check(B, q, seq, pos, 8, 1, 1)
    # (row 4: scores past the fp32 range are as large, and the lower index goes first)
    assert all({20, 50} <= set(got[r, h]) for r in (0, 1, 2, 3, 5) for h in range(2))
    assert got[1, 0].tolist() == [0, 1, 2, 3, 4, 20, 50, 124]


def test_selection_flags_what_is_out_of_range(B):
    from paged_kv_cache_96_gb300 import binding as L
    x = Bounds([500, 300], 1, 64, 16, seed=2)
    q = query(2, 4, 64, torch.float16)
    for seq, pos in (([2, 1], [5, 299]), ([0, 1], [-1, 299]),
                     ([0, 1], [x.tables.shape[1] * 16, 299])):
        x.err.zero_()
        got = x.select(B, q, seq, pos, 5, 1, 1, max_ctx=10000)
        assert int(x.err.item()) == L.DEVERR_TOKEN_RANGE
        assert (got[0] == -1).all() and got[1, 0, -1] == 18
    x.err.zero_()
    got = x.select(B, q, [0, 1], [499, 299], 5, 1, 1, max_ctx=320)     # clipped: 20 blocks
    assert int(x.err.item()) == L.DEVERR_CONTEXT_RANGE
    assert got[0, 0, -1] == 19 and got[1, 0, -1] == 18
    x.err.zero_()
    bad = x.tables.copy()
    bad[0, 3], bad[0, 9] = x.N, -4
    got = x.select(B, q, [0, 1], [499, 299], 5, 1, 1, tables=bad)
    assert int(x.err.item()) == L.DEVERR_BLOCK_RANGE
    assert not {3, 9} & set(got[0, 0].tolist())


def test_selection_repeats_and_takes_any_stream(B):
    x = Bounds([30000, 9000], 4, 128, 16, seed=12)
    q = query(2, 16, 128, torch.bfloat16)
    a = x.check(B, q, [0, 1], [29999, 8999], 64, 1, 2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = x.select(B, q, [0, 1], [29999, 8999], 64, 1, 2)
    c = x.select(B, q, [0, 1], [29999, 8999], 64, 1, 2, stream=side)
    assert np.array_equal(a, b) and np.array_equal(a, c)


def test_blocks_past_32_bits(B):
    """Codes and keys whose bytes lie past 4 GB of their pools."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("not enough memory")
    N, K, D, bs = 2_200_000, 8, 128, 16
    codes = torch.zeros((N, K, 2, D), dtype=torch.int8, device="cuda")
    scales = torch.ones((N, K), device="cuda")
    tables = np.array([[N - 1 - 3 * j for j in range(40)]])
    for j, level in ((7, 90), (23, 100), (24, 80)):
        codes[int(tables[0, j]), :, 1] = level
    q = torch.ones((1, 16, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full((1, K, 4), 9, dtype=torch.int32, device="cuda")
    B.pa_select_blocks(out, q, codes, scales, i32(tables), i32([0]), i32([639]), 640, bs, 0, 1)
    assert out.tolist() == [[[7, 23, 24, 39]] * K]
    del codes, scales
    N, K = 40000, 32
    keys = torch.zeros((N, bs, K, D), dtype=torch.bfloat16, device="cuda")
    keys[N - 1, 3, :, 5] = -2.0
    codes = torch.full((N, K, 2, D), 1, dtype=torch.int8, device="cuda")
    scales = torch.full((N, K), 3.0, device="cuda")
    B.pa_summarize_blocks(codes, scales, keys, i32([[N - 1, N - 2]]), i32([20]))
    assert codes[N - 1, :, 0, 5].eq(-127).all() and codes[N - 1].ne(0).sum() == K
    assert scales[N - 2].eq(0).all() and scales[N - 3].eq(3).all()
    assert torch.equal(scales[N - 1], torch.full((K,), 2.0, device="cuda") *
                       torch.tensor(1 / 127.0, device="cuda"))


def test_the_longest_contexts(B):
    """300,000 blocks of one context at lists of 128, beside a short one; more than the
    shared memory of eight CTAs holds is refused."""
    N, D, bs = 300_000, 64, 16
    codes = torch.zeros((N, 2, 2, D), dtype=torch.int8, device="cuda")
    scales = torch.ones((N, 2), device="cuda")
    best = [0, 7, 1000, 123_456, 262_143, 262_144, 299_000]
    for j, b in enumerate(best):
        codes[b, 1, 1] = 100 - j
    tables = torch.arange(N, dtype=torch.int32, device="cuda").expand(2, N).contiguous()
    q = torch.ones((2, 4, D), dtype=torch.float16, device="cuda")
    out = torch.full((2, 2, 128), 9, dtype=torch.int32, device="cuda")
    B.pa_select_blocks(out, q, codes, scales, tables, i32([0, 1]), i32([N * bs - 1, 40]), N * bs, bs,
                       0, 1)
    # (of equal scores the lower blocks)
    rest = [b for b in range(200) if b not in best][:127 - len(best)]
    assert out[0, 1].tolist() == sorted(best + rest) + [N - 1]
    assert out[0, 0].tolist() == list(range(127)) + [N - 1]
    assert out[1].tolist() == [[0, 1, 2] + [-1] * 125] * 2
    wide = torch.zeros((2, 500_000), dtype=torch.int32, device="cuda")
    with pytest.raises(B.PAError) as e:
        B.pa_select_blocks(out, q, codes, scales, wide, i32([0, 1]), i32([9, 9]), 500_000 * bs, bs,
                           0, 1)
    assert e.value.status == B.PA_ERR_UNSUPPORTED
