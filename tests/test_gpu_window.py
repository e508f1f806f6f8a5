"""Windowed decode and chunked attention against the definition in 64 bits.

Pools hold NaN wherever no visible token is (spare blocks, rows past the
context, blocks that the window has left, hidden rows beside visible ones), and
table entries of blocks without a visible token point outside the pool."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import operator_refs as R  # noqa: E402

SCALE = 0.02


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


class Case:
    def __init__(self, ctx, rows, H, K, D, bs, dtype, fp8, window, sinks, seed=0, poison=True,
                 amp=1.0):
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.rows = np.asarray(ctx), np.asarray(rows)
        self.window, self.sinks, self.dtype, self.fp8 = window, sinks, dtype, fp8
        S, T = len(ctx), int(self.rows.sum())
        self.start = np.concatenate([[0], np.cumsum(self.rows)])
        blocks = -(-self.ctx // bs)
        N, MB = int(blocks.sum()) + 3, max(1, int(blocks.max()))
        ids = r.permutation(N)
        tables = np.full((S, MB), N + 5, dtype=np.int32)   # outside the pool: never looked at
        live = np.zeros((N, bs), dtype=bool)
        at = 0
        for s in range(S):
            mine = ids[at:at + blocks[s]]
            at += blocks[s]
            first = self.ctx[s] - max(1, self.rows[s])      # position of the first row
            low = max(0, first + 1 - window)
            p = np.arange(self.ctx[s])
            seen = p[(p >= low) | (p < sinks)] if poison else p
            tables[s, seen // bs] = mine[seen // bs]
            live[mine[seen // bs], seen % bs] = True
        shape = (N, bs, K, D)
        k, v = (torch.randn(shape, generator=g) * amp for _ in range(2))
        hide = torch.as_tensor(~live)[..., None, None].expand(shape)
        if fp8:
            kc, vc = ((x / SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                      for x in (k, v))
            kc, vc = (x.masked_fill(hide, 0x7F) for x in (kc, vc))
        else:
            kc, vc = (x.to(dtype).masked_fill(hide, float("nan")) for x in (k, v))
        self.kc, self.vc = kc.cuda(), vc.cuda()
        self.tables = tables
        self.q = (torch.randn((T, H, D), generator=g)).to(dtype).cuda()
        self.out = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
        i = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.d_tables, self.d_ctx, self.d_start = i(tables), i(ctx), i(self.start)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale, self.kv = D ** -0.5, SCALE if fp8 else 1.0
        self.max_ctx = int(self.ctx.max())

    def decode(self, B, P=0, ws=None, **kw):
        S, H, D = self.q.shape
        K = self.kc.shape[2]
        n = B.pa_window_workspace_bytes(S, H, K, D, self.max_ctx, self.window, self.sinks, P)
        if ws is None and n:
            ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        B.pa_decode_attention_window(self.out, self.q, self.kc, self.vc, self.d_tables, self.d_ctx,
                                     self.max_ctx, self.scale, self.window, self.sinks, P, ws,
                                     k_scale=self.kv, v_scale=self.kv, error_word=self.err, **kw)

    def chunk(self, B, **kw):
        B.pa_prefill_attention_window(self.out, self.q, self.kc, self.vc, self.d_tables,
                                      self.d_start, self.d_ctx, self.max_ctx, self.scale,
                                      self.window, self.sinks, k_scale=self.kv, v_scale=self.kv,
                                      error_word=self.err, **kw)

    def check(self, what=""):
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        kc, vc = (R.pool_values(x, self.kv) for x in (self.kc, self.vc))
        want, tol = R.window_attention(self.q, kc, vc, self.tables, self.start, self.ctx,
                                       self.scale, self.window, self.sinks, self.dtype,
                                       torch.float16 if self.fp8 else self.dtype)
        R.assert_within(self.out, want, tol, what)


TYPES = [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
         (torch.float16, True)]
IDS = ["bf16", "f16", "bf16-fp8", "f16-fp8"]

DECODE = [
    # H, K, D, bs, window, sinks, contexts
    (4, 4, 64, 16, 128, 4, [1, 2, 15, 16, 17, 500]),
    (8, 2, 128, 16, 1, 0, [1, 16, 17, 33, 100]),
    (8, 1, 128, 16, 16, 0, [1, 15, 16, 17, 31, 32, 33, 300]),
    (16, 1, 64, 32, 33, 1, [1, 33, 34, 35, 64, 65, 200]),
    (10, 2, 128, 64, 100, 16, [5, 100, 116, 117, 130, 1000]),
    (3, 1, 128, 16, 50, 17, [50, 66, 67, 68, 83, 84, 500]),
    (32, 2, 128, 256, 300, 255, [300, 555, 556, 900, 2000]),
    (9, 1, 64, 16, 7, 128, [1, 128, 135, 136, 151, 152, 400]),
    (4, 1, 128, 16, 5000, 3, [1, 700, 1300]),                # a window past every context
    (4, 1, 64, 16, 1, 5000, [1, 100, 333]),                  # first tokens past every context
]


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("H,K,D,bs,window,sinks,ctx", DECODE)
def test_decode(B, dtype, fp8, H, K, D, bs, window, sinks, ctx):
    c = Case(ctx, [1] * len(ctx), H, K, D, bs, dtype, fp8, window, sinks, seed=window + D)
    for P in (0, 16, 32, 48, 256):
        c.out.fill_(7.0)
        c.decode(B, P)
        c.check(f"P={P}")


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_decode_every_border(B, dtype, fp8):
    """Every place of the window's start and of the context's end in a tile."""
    for window, sinks in ((40, 0), (40, 5), (17, 16), (64, 31)):
        c = Case(range(60, 60 + 35), [1] * 35, 4, 2, 64, 16, dtype, fp8, window, sinks, seed=window)
        c.decode(B)
        c.check()


def test_decode_many_partials(B):
    """Past eight partitions the reduce kernel merges; its lengths are compact
    ones, and one workspace serves calls of both kinds in turn."""
    c = Case([3000, 700, 5, 1400], [1] * 4, 8, 2, 128, 16, torch.bfloat16, False, 600, 20)
    n = B.pa_window_workspace_bytes(4, 8, 2, 128, 3000, 600, 20, 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for P in (16, 80, 16, 320, 64):
        c.out.fill_(7.0)
        c.decode(B, P, ws)
        c.check(f"P={P}")
    assert int(ws[:1 << 20].sum().item()) == 0


def test_wide_window_is_plain_decode(B):
    c = Case([700, 33, 1, 256], [1] * 4, 16, 2, 128, 16, torch.bfloat16, False, 4096, 0)
    plain = torch.empty_like(c.out)
    c.decode(B)
    B.pa_decode_attention(plain, c.q, c.kc, c.vc, c.d_tables, c.d_ctx, c.max_ctx, c.scale)
    torch.cuda.synchronize()
    assert torch.equal(plain, c.out)


CHUNK = [
    # H, K, D, bs, window, sinks, contexts, rows
    (8, 2, 64, 16, 33, 3, [37, 70, 50, 30], [1, 1, 50, 30]),
    (4, 4, 128, 16, 1, 0, [5, 130], [5, 130]),
    (8, 1, 128, 16, 16, 0, [300, 33], [64, 33]),
    (16, 1, 128, 32, 100, 16, [700, 128, 1], [300, 128, 1]),
    (3, 1, 64, 16, 200, 17, [400, 150], [171, 149]),        # group does not divide 128
    (2, 2, 128, 64, 64, 64, [1000, 64], [200, 60]),
    (10, 2, 128, 16, 130, 200, [900, 201, 199], [129, 100, 199]),
    (4, 1, 128, 16, 5000, 3, [600], [600]),                 # a window past every context
    (4, 1, 64, 16, 8, 5000, [300], [200]),
    (1, 1, 64, 256, 60, 1, [513], [512]),
]


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("H,K,D,bs,window,sinks,ctx,rows", CHUNK)
def test_chunk(B, dtype, fp8, H, K, D, bs, window, sinks, ctx, rows):
    c = Case(ctx, rows, H, K, D, bs, dtype, fp8, window, sinks, seed=window + D)
    c.chunk(B)
    c.check()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_chunk_every_border(B, dtype, fp8):
    for window, sinks, n in ((40, 0, 20), (70, 5, 3), (17, 16, 33)):
        ctx = list(range(100, 100 + 35))
        c = Case(ctx, [n] * 35, 4, 2, 64, 16, dtype, fp8, window, sinks, seed=window)
        c.chunk(B)
        c.check()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_chunk_many_units(B, dtype, fp8):
    """More row tiles than one round of the grid: the ordered deal and the query
    tiles by TMA."""
    ctx = [900, 100, 641, 300] * 6
    c = Case(ctx, [90, 100, 64, 77] * 6, 32, 16, 64, 16, dtype, fp8, 90, 5, seed=3)
    c.chunk(B)
    c.check()


def test_chunk_of_one_row_is_decode(B):
    ctx = [1, 40, 333, 1000]
    c = Case(ctx, [1] * 4, 8, 2, 128, 16, torch.bfloat16, False, 100, 6)
    c.chunk(B)
    c.check()
    c.out.fill_(7.0)
    c.decode(B)
    c.check()


def test_wide_window_is_plain_prefill(B):
    c = Case([300, 77], [200, 77], 8, 2, 128, 16, torch.bfloat16, False, 4096, 0)
    plain = torch.empty_like(c.out)
    c.chunk(B)
    B.pa_prefill_attention(plain, c.q, c.kc, c.vc, c.d_tables, c.d_start, c.d_ctx, c.max_ctx,
                           c.scale)
    torch.cuda.synchronize()
    assert (plain.float() - c.out.float()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_bad_lengths_and_tables(B, call):
    """Clipped and flagged, never followed: contexts past the table or negative,
    table entries outside the pool, offsets outside the rows."""
    mk = lambda: Case([200, 100, 90], [1] * 3, 8, 2, 128, 16, torch.bfloat16, False, 64, 4)  # noqa: E731
    c = mk()
    c.d_ctx[0] = 10 ** 9
    getattr(c, call)(B)
    torch.cuda.synchronize()
    assert int(c.err.item()) & B.DEVERR_CONTEXT_RANGE
    c = mk()
    c.d_ctx[1] = -3
    getattr(c, call)(B)
    torch.cuda.synchronize()
    assert int(c.err.item()) == B.DEVERR_CONTEXT_RANGE
    assert (c.out[1] == 0).all()
    for bad in (-1, c.kc.shape[0], 2 ** 31 - 1):
        c = mk()
        c.d_tables[2, 90 // 16] = bad
        getattr(c, call)(B)
        torch.cuda.synchronize()
        assert int(c.err.item()) == B.DEVERR_BLOCK_RANGE
        assert torch.isfinite(c.out[:2].float()).all()


def test_chunk_rows_past_the_last_and_odd_offsets(B):
    c = Case([200, 100], [20, 30], 8, 2, 128, 16, torch.bfloat16, False, 64, 4)
    big_q = torch.cat([c.q, c.q])
    big_out = torch.full_like(big_q, 7.0)
    q, out = c.q, c.out
    c.q, c.out = big_q, big_out
    c.chunk(B)
    torch.cuda.synchronize()
    assert (big_out[50:] == 7).all()          # rows of no sequence are left
    c.q, c.out = q, big_out[:50]
    c.check()
    c.q, c.out = big_q, torch.full_like(big_q, 7.0)
    c.d_start[2] = 10 ** 6                    # past the rows: clipped, flagged
    c.chunk(B)
    torch.cuda.synchronize()
    assert int(c.err.item()) & B.DEVERR_TOKEN_RANGE
    c.d_start.copy_(torch.tensor([-5, 20, 10]))
    c.chunk(B)
    torch.cuda.synchronize()
    assert int(c.err.item()) & B.DEVERR_TOKEN_RANGE


def test_chunk_longer_than_its_context(B):
    """Rows at negative positions get zeros, the others their answer."""
    c = Case([10, 40], [16, 40], 4, 2, 64, 16, torch.float16, False, 12, 2, poison=False)
    c.chunk(B)
    c.check()
    assert (c.out[:6] == 0).all()


def test_context_zero(B):
    c = Case([5, 40], [1, 1], 4, 2, 64, 16, torch.float16, False, 12, 2)
    c.d_ctx[0] = 0
    c.decode(B)
    torch.cuda.synchronize()
    assert (c.out[0] == 0).all() and torch.isfinite(c.out[1].float()).all()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("H,K,D,window,sinks", [(8, 2, 128, 40, 5), (4, 4, 64, 20, 0),
                                               (6, 2, 64, 500, 2)])
def test_chunk_values_hidden_from_some_rows(B, dtype, fp8, H, K, D, window, sinks):
    """Infinite and NaN values at positions that some rows of a chunk see and
    others do not: each row has what the definition gives it, element by
    element."""
    c = Case([300, 90], [130, 90], H, K, D, 16, dtype, fp8, window, sinks, seed=8)
    kc, vc = c.kc, c.vc
    spots = [(0, 200, 0, 3), (0, 290, K - 1, 5), (0, 171, 0, D - 1), (1, 60, 0, 9), (1, 0, 0, 1)]
    for s, p, h, d in spots:
        b, r = c.tables[s][p // 16], p % 16
        if b >= vc.shape[0]:
            continue  # (no row sees it)
        if fp8:
            vc[b, r, h, d] = 0x7F
        else:
            vc[b, r, h, d] = float("inf") if d % 2 else float("nan")
    c.chunk(B)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    got = c.out.double().cpu().numpy()
    kv, vv = (R.pool_values(x, c.kv) for x in (kc, vc))
    hot = ~np.isfinite(vv)
    # the definition: an element is non-finite where a value the row sees is
    clean = np.where(hot, 0.0, vv)
    want, tol = R.window_attention(c.q, kv, clean, c.tables, c.start, c.ctx, c.scale, window, sinks,
                                   dtype, torch.float16 if fp8 else dtype)
    touched = np.zeros(want.shape, dtype=bool)
    for s in range(2):
        for i in range(int(c.rows[s])):
            pos = int(c.ctx[s] - c.rows[s] + i)
            p = R.visible(pos, int(c.ctx[s]), window, sinks)
            bad = hot[c.tables[s][p // 16], p % 16].any(0)        # [K, D]
            touched[c.start[s] + i] = np.repeat(bad, H // K, axis=0)
    assert touched.any() and not touched.all()
    assert np.array_equal(~np.isfinite(got), touched)
    assert (np.abs(got - want) <= tol)[~touched].all()


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_value_hidden_from_rows_of_a_long_context(B, fp8):
    """Rows before a NaN value share tiles with rows that see it: they are
    computed anew from 40,000 keys, which must not run out another role's wait
    (here 5 ms) nor change the units after them."""
    c = Case([40000, 70], [64, 70], 4, 1, 128, 64, torch.bfloat16, fp8, 60000, 0, seed=4)
    pos, d = 40000 - 64 + 16, 7
    c.vc[c.tables[0][pos // 64], pos % 64, 0, d] = 0x7F if fp8 else float("nan")
    B.pa_set_stage_wait_limit_ns(5_000_000)
    try:
        c.chunk(B)
        torch.cuda.synchronize()
    finally:
        B.pa_set_stage_wait_limit_ns(0)
    assert int(c.err.item()) == 0
    kv, vv = (R.pool_values(x, c.kv) for x in (c.kc, c.vc))
    want, tol = R.window_attention(c.q, kv, np.where(np.isfinite(vv), vv, 0.0), c.tables, c.start,
                                   c.ctx, c.scale, c.window, c.sinks, torch.bfloat16,
                                   torch.float16 if fp8 else torch.bfloat16)
    got = c.out.double().cpu().numpy()
    sees = np.zeros(got.shape, dtype=bool)
    sees[16:64, :, d] = True
    assert np.array_equal(~np.isfinite(got), sees)
    assert (np.abs(got - want) <= tol)[~sees].all()


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_hidden_values_in_the_last_of_many_units(B, fp8):
    """More units a CTA than it keeps in shared memory; NaN values in the first and
    last of them."""
    T, H, D, bs, W, dtype = 210000, 16, 64, 16, 9, torch.float16
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty((T, H, D), dtype=dtype, device="cuda").normal_(generator=g)
    n = -(-T // bs)
    kc, vc = (torch.empty((n, bs, 1, D), device="cuda").normal_(generator=g) for _ in range(2))
    kc, vc = (x.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(dtype)
              for x in (kc, vc))
    spots = [(5, 3), (70003, 8), (T - 12, 60)]
    for pos, d in spots:
        vc[pos // bs, pos % bs, 0, d] = 0x7F if fp8 else float("nan")
    i = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    out, err = torch.full_like(q, 7), i([0])
    B.pa_prefill_attention_window(out, q, kc, vc, i(np.arange(n))[None], i([0, T]), i([T]), T,
                                  0.125, W, 0, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    sees = torch.zeros_like(out, dtype=torch.bool)
    for pos, d in spots:
        sees[pos:pos + W, :, d] = True
    assert torch.equal(~torch.isfinite(out), sees)
    kv, vv = (R.pool_values(x) for x in (kc, vc))
    vv = np.where(np.isfinite(vv), vv, 0.0)
    for pos, _ in spots:  # rows about each of them
        lo, hi = max(0, pos - 20), min(T, pos + 20)
        want, tol = R.window_attention(q[lo:hi], kv, vv, np.arange(n)[None], [0, hi - lo], [hi],
                                       0.125, W, 0, dtype, dtype)
        far = np.abs(out[lo:hi].double().cpu().numpy() - want)
        assert (far <= tol)[~sees[lo:hi].cpu().numpy()].all()


@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_large_scores(B, call):
    """Scores in the hundreds: one key takes nearly all the weight."""
    c = Case([500, 77], [1, 1], 8, 2, 128, 16, torch.bfloat16, False, 100, 4, amp=20.0, seed=5)
    getattr(c, call)(B)
    c.check()


def test_captured_and_on_another_stream(B):
    c = Case([500, 77, 300], [1, 1, 1], 8, 2, 128, 16, torch.bfloat16, False, 100, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = B.pa_window_workspace_bytes(3, 8, 2, 128, 500, 100, 4, 32)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    c.decode(B, 32, ws, stream=side)
    torch.cuda.synchronize()
    c.check()
    for call in ("decode", "chunk"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.decode(B, 32, ws) if call == "decode" else c.chunk(B)
        for _ in range(3):
            c.out.fill_(7.0)
            g.replay()
            c.check(call)


@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_stage_wait_limit(B, call):
    """A fill that never comes ends in a flag, and the next call is whole."""
    c = Case([500, 77, 300], [1, 1, 1], 8, 2, 128, 16, torch.bfloat16, False, 100, 4)
    B.pa_set_stage_wait_limit_ns(2_000_000)
    B.pa_debug_withhold_first_fill(True)
    try:
        getattr(c, call)(B)
        torch.cuda.synchronize()
    finally:
        B.pa_debug_withhold_first_fill(False)
        B.pa_set_stage_wait_limit_ns(0)
    assert int(c.err.item()) == B.DEVERR_TIMEOUT
    c.err.zero_()
    c.out.fill_(7.0)
    getattr(c, call)(B)
    c.check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_stage_wait_limit_over_codes(B, call, D):
    """The same where the fill that never comes is one of FP8 codes."""
    c = Case([500, 77, 300], [1, 1, 1], 8, 2, D, 32, torch.bfloat16, True, 100, 4)
    B.pa_set_stage_wait_limit_ns(2_000_000)
    B.pa_debug_withhold_first_fill(True)
    try:
        getattr(c, call)(B)
        torch.cuda.synchronize()
    finally:
        B.pa_debug_withhold_first_fill(False)
        B.pa_set_stage_wait_limit_ns(0)
    assert int(c.err.item()) == B.DEVERR_TIMEOUT
    c.err.zero_()
    c.out.fill_(7.0)
    getattr(c, call)(B)
    c.check()


def test_far_context(B):
    """A context of 400,000 tokens whose blocks but the visible ones are gone."""
    c = Case([400000, 33], [1, 1], 8, 2, 128, 16, torch.bfloat16, False, 200, 9)
    c.decode(B)
    c.check()
    c = Case([400000, 33], [70, 33], 8, 2, 128, 16, torch.bfloat16, False, 200, 9)
    c.chunk(B)
    c.check()


@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_binding_checks_every_tensor(B, call):
    """Type, device, layout and range of each argument, and what is taken: NumPy
    numbers, windows past 32 bits, a stream object, an error word or none."""
    c = Case([40, 70], [1, 1], 4, 2, 64, 16, torch.float16, False, 9, 2, poison=False)
    run = getattr(c, call)
    for name, bad, error in (
            ("q", c.q.float(), TypeError), ("q", c.q.cpu(), ValueError),
            ("q", c.q.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
            ("q", c.q[0], ValueError), ("out", c.out.bfloat16(), TypeError),
            ("out", c.out.cpu(), ValueError), ("out", c.out[:1], ValueError),
            ("kc", c.kc.bfloat16(), TypeError), ("kc", c.kc[:, ::2], ValueError),
            ("vc", c.vc[:-1], ValueError), ("vc", c.vc.cpu(), ValueError),
            ("d_tables", c.d_tables.long(), TypeError), ("d_tables", c.d_tables[:1], ValueError),
            ("d_ctx", c.d_ctx.cpu(), ValueError), ("d_ctx", c.d_ctx.float(), TypeError),
            ("err", c.err.long(), TypeError), ("err", c.err.cpu(), ValueError),
            ("max_ctx", 1 << 40, ValueError),
            ("scale", "large", TypeError), ("scale", float("inf"), B.PAError)):
        good = getattr(c, name)
        setattr(c, name, bad)
        with pytest.raises(error):
            run(B)
        setattr(c, name, good)
    with pytest.raises(AttributeError):
        run(B, stream=3)
    assert bool((c.out == 7).all())
    c.window, c.sinks, c.max_ctx = 1 << 40, np.int64(2), np.int32(c.max_ctx)
    run(B, stream=torch.cuda.current_stream())
    c.window = 70                       # what a window past every context is
    c.check()
    c.err = None
    c.out.fill_(7)
    run(B)
    c.err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check()
