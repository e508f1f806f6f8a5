"""Windowed attention where keys, queries or values are not numbers or infinite, and
its outputs from call to call.  The definition in 64 bits says for every element
whether it is a number, which infinity, or not a number."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import operator_refs as R  # noqa: E402
from test_gpu_window import IDS, TYPES, Case  # noqa: E402

FLOATS = [(torch.bfloat16, False), (torch.float16, False)]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


def definition(c):
    """Outputs and tolerances of a Case as operator_refs.window_attention has them,
    for pools and queries that may hold infinities and NaN: a key whose score is -inf
    has weight 0 and no share in the scores' rounding."""
    q = c.q.double().cpu().numpy()
    kc, vc = (R.pool_values(x, c.kv) for x in (c.kc, c.vc))
    T, H, D = q.shape
    bs, K = kc.shape[1], kc.shape[2]
    G = H // K
    p_half = R.HALF_STEP[torch.float16 if c.fp8 else c.dtype]
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    with np.errstate(all="ignore"):
        for s, n in enumerate(c.ctx):
            n, lo, hi = int(n), int(c.start[s]), int(c.start[s + 1])
            for r in range(lo, hi):
                pos = n - (hi - lo) + (r - lo)
                if pos < 0:
                    continue
                p = R.visible(pos, n, c.window, c.sinks)
                blk = c.tables[s][p // bs]
                for h in range(K):
                    k, v = kc[blk, p % bs, h], vc[blk, p % bs, h]
                    real = np.isfinite(k).all(-1)
                    for g in range(h * G, (h + 1) * G):
                        x = (k * q[r, g]).sum(-1) * c.scale
                        w = np.exp(x - x.max())
                        w = (w / w.sum())[:, None]
                        o = np.where(w == 0, np.where(np.isfinite(v), 0.0, np.nan), w * v).sum(0)
                        size = c.scale * (np.abs(k[real]) @ np.abs(q[r, g])).max(initial=0)
                        e = 2 * ((D + 4) * 2.0 ** -22 * size + (len(p) + 8) * 2.0 ** -23)
                        mass = (w * np.abs(np.where(np.isfinite(v), v, 0))).sum(0)
                        out[r, g] = o
                        tol[r, g] = (R.HALF_STEP[c.dtype] * np.abs(o) +
                                     1.01 * (p_half + e) * mass + 2.0 ** -24)
    return out, tol


def check(c, what=""):
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0, what
    got = c.out.double().cpu().numpy()
    want, tol = definition(c)
    wrong = int((np.isnan(got) != np.isnan(want)).sum())
    assert wrong == 0, f"{what}: {wrong} elements numbers on one side only"
    for sign in (1, -1):
        wrong = int(((got == sign * np.inf) != (want == sign * np.inf)).sum())
        assert wrong == 0, f"{what}: {wrong} infinities on one side only"
    real = np.isfinite(want)
    far = np.abs(got[real] - want[real])
    assert (far <= tol[real]).all(), f"{what}: worst {np.max(far / tol[real]):.2f}x"
    return want


def place(c, s, p):
    """Block and row of position p of sequence s."""
    bs = c.kc.shape[1]
    return int(c.tables[s][p // bs]), p % bs


def put(c, pool, s, positions, d, value):
    for p in positions:
        pool[place(c, s, p)][..., d] = value


PARTITIONS = (0, 144, 96, 80, 64, 32, 16)  # of 288 tokens: 1, 2, 3, 4, 5, 9 and 18


@pytest.mark.parametrize("dtype,fp8", FLOATS, ids=IDS[:2])
@pytest.mark.parametrize("H,K,D", [(8, 2, 128), (16, 1, 64), (3, 3, 64)])
@pytest.mark.parametrize("span", [(0, 144), (144, 288), (80, 240)])
def test_decode_partition_of_keys_without_weight(B, dtype, fp8, H, K, D, span):
    """Keys whose scores are all -inf, a partition and more of them: they have weight 0
    whatever the partition size, and the others their own."""
    c = Case([288, 30, 288], [1] * 3, H, K, D, 16, dtype, fp8, 5000, 0, seed=7)
    c.q[..., 1] = c.q[..., 1].abs() + 0.5
    put(c, c.kc, 0, range(*span), 1, float("-inf"))
    for P in PARTITIONS:
        c.out.fill_(7.0)
        c.decode(B, P)
        check(c, f"P={P}")


@pytest.mark.parametrize("dtype,fp8", FLOATS, ids=IDS[:2])
@pytest.mark.parametrize("window,sinks", [(17, 3), (33, 0), (50, 16)])
def test_decode_border_tile_without_weight(B, dtype, fp8, window, sinks):
    """Partitions of one tile, whose few visible keys (the first tokens' or the
    window's oldest) have a score of -inf."""
    c = Case(range(100, 117), [1] * 17, 4, 2, 64, 16, dtype, fp8, window, sinks, seed=9)
    c.q[..., 1] = c.q[..., 1].abs() + 0.5
    for s, n in enumerate(c.ctx):
        low = int(n) - window
        put(c, c.kc, s, [*range(sinks), *range(low, -(-(low + 1) // 16) * 16)], 1, float("-inf"))
    for P in (0, 16, 32):
        c.out.fill_(7.0)
        c.decode(B, P)
        check(c, f"P={P}")


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("span", [(0, 144), (144, 288), (80, 240), (100, 101)])
def test_decode_partition_of_keys_that_are_not_numbers(B, dtype, fp8, span):
    """A visible key that is not a number makes its row so, also where a whole
    partition holds nothing else."""
    c = Case([288, 30, 288], [1] * 3, 8, 2, 128, 16, dtype, fp8, 5000, 0, seed=7)
    put(c, c.kc, 0, range(*span), 5, 0x7F if fp8 else float("nan"))
    for P in PARTITIONS:
        c.out.fill_(7.0)
        c.decode(B, P)
        want = check(c, f"P={P}")
    assert np.isnan(want[0]).all() and np.isfinite(want[1:]).all()


@pytest.mark.parametrize("dtype,fp8", FLOATS, ids=IDS[:2])
@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_rows_whose_scores_are_all_minus_infinity(B, dtype, fp8, call):
    """Their softmax is not a number; rows that see one key more have their answer."""
    rows = [1, 1] if call == "decode" else [45, 50]
    c = Case([200, 50], rows, 8, 2, 128, 16, dtype, fp8, 20, 0, seed=3, poison=False)
    c.q[..., 1] = c.q[..., 1].abs() + 0.5
    put(c, c.kc, 0, range(175, 200), 1, float("-inf"))
    for P in (0, 16) if call == "decode" else (0,):
        c.out.fill_(7.0)
        c.decode(B, P) if call == "decode" else c.chunk(B)
        want = check(c, f"P={P}")
    bad = np.isnan(want).all((1, 2))
    assert bad[:rows[0]].sum() == min(rows[0], 6) and not bad[rows[0]:].any()


def timed(run):
    run()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    run()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_of_a_diverged_sequence_takes_no_longer(B, fp8):
    """Rows that are not numbers by what they see -- a query, a key, an old value -- are
    the definition's and need nothing computed anew, however long their context."""
    def make():
        return Case([40000, 70], [64, 70], 4, 1, 128, 64, torch.bfloat16, fp8, 60000, 0, seed=4)
    nan = 0x7F if fp8 else float("nan")
    c = make()
    clean = timed(lambda: c.chunk(B))
    whole = c.out.clone()
    assert torch.isfinite(whole.float()).all()
    for what in ("query", "key", "value"):
        c = make()
        bad = torch.zeros_like(whole, dtype=torch.bool)
        if what == "query":
            c.q[3:50, 1, 7] = float("nan")
            bad[3:50, 1] = True
        elif what == "key":
            put(c, c.kc, 0, [1234], 9, nan)
            bad[:64] = True
        else:
            put(c, c.vc, 0, [1234], 9, nan)
            bad[:64, :, 9] = True
        ms = timed(lambda: c.chunk(B))
        assert int(c.err.item()) == 0
        assert torch.equal(torch.isnan(c.out), bad), what
        assert torch.equal(c.out[~bad], whole[~bad]), what
        assert ms < 3 * clean + 0.5, f"{what}: {ms:.2f} ms, {clean:.2f} ms without"


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_chunk_rows_before_the_first_beside_values_that_are_not_numbers(B, dtype, fp8):
    """Rows at negative positions stay zero beside rows that see such a value."""
    for window, sinks in ((12, 2), (100, 0)):
        c = Case([10, 40], [16, 40], 4, 2, 64, 16, dtype, fp8, window, sinks, poison=False)
        put(c, c.vc, 0, [5], 3, 0x7F if fp8 else float("nan"))
        if not fp8:
            put(c, c.vc, 0, [7], 11, float("inf"))
        c.chunk(B)
        check(c)
        assert (c.out[:6] == 0).all()


@pytest.mark.parametrize("dtype,fp8", FLOATS, ids=IDS[:2])
@pytest.mark.parametrize("H,K,D,window,sinks", [(8, 2, 128, 40, 5), (4, 4, 64, 20, 0),
                                               (6, 2, 64, 500, 2)])
def test_chunk_infinite_values_beside_hidden_ones(B, dtype, fp8, H, K, D, window, sinks):
    """What a row sees says which infinity an element is; a NaN or another infinity at the
    same element of a key hidden from the row says nothing."""
    c = Case([300, 90], [130, 90], H, K, D, 16, dtype, fp8, window, sinks, seed=8, poison=False)
    inf, nan = float("inf"), float("nan")
    for s, p, d, x in ((0, 200, 3, inf), (0, 210, 3, nan), (0, 205, 7, -inf), (0, 230, 7, inf),
                       (0, 260, 9, nan), (0, 263, 9, inf), (0, 171, D - 1, inf),
                       (0, 173, D - 1, inf), (1, 0, 1, -inf), (1, 60, 1, nan), (1, 33, 2, inf)):
        put(c, c.vc, s, [p], d, x)
    c.chunk(B)
    want = check(c)
    assert (want == inf).any() and (want == -inf).any() and np.isnan(want).any()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
def test_outputs_repeat_bit_by_bit(B, dtype, fp8):
    """The same call again has the same bits, whichever CTA merges its partials."""
    c = Case([3000, 700, 5, 1400], [1] * 4, 8, 2, 128, 16, dtype, fp8, 600, 20)
    d = Case([900, 100, 641, 300] * 4, [90, 100, 64, 77] * 4, 32, 8, 64, 16, dtype, fp8, 90, 5)
    for P in (0, 16, 80, 224, 320):
        c.decode(B, P)
        first = c.out.clone()
        for _ in range(8):
            c.out.fill_(7.0)
            c.decode(B, P)
            assert torch.equal(first, c.out), P
    d.chunk(B)
    first = d.out.clone()
    for _ in range(8):
        d.out.fill_(7.0)
        d.chunk(B)
        assert torch.equal(first, d.out)
    c.check()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20, 1 << 40])
def test_chunk_longer_than_its_context_behind_a_window_past_every_length(B, dtype, fp8, window):
    """Rows at negative positions, whose window would start before -2^31."""
    c = Case([10, 40, 0], [300, 40, 9], 4, 2, 64, 16, dtype, fp8, 5000, 2, poison=False)
    c.window = window
    c.chunk(B)
    c.window = 5000     # what a window past every context is
    check(c)
    assert (c.out[:290] == 0).all() and (c.out[340:] == 0).all()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("call", ["decode", "chunk"])
@pytest.mark.parametrize("scale", [1e-39, 1e-44, 1.5e-38])
def test_scales_below_the_normal_range(B, dtype, fp8, call, scale):
    """Every visible key has the same weight, hidden ones none."""
    rows = [1, 1] if call == "decode" else [45, 30]
    c = Case([100, 30], rows, 8, 2, 64, 16, dtype, fp8, 20, 3, seed=6)
    c.scale = scale
    getattr(c, call)(B)
    check(c)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs", [3, 300, 600])
def test_chunk_offsets_that_go_back(B, fp8, seqs):
    """Offsets that decrease name rows twice: flagged, and no row past the last one is
    written, however many rows they add up to."""
    c = Case([90] * seqs, [40] * seqs, 8, 2, 128, 16, torch.bfloat16, fp8, 30, 2, poison=False)
    T = 60
    c.q, c.out = c.q[:T], torch.full((T + 50, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    whole, c.out = c.out, c.out[:T]
    c.d_start.copy_(torch.arange(seqs + 1, dtype=torch.int32) % 2 * T)
    c.chunk(B)
    torch.cuda.synchronize()
    assert int(c.err.item()) == B.DEVERR_TOKEN_RANGE
    assert (whole[T:] == 7).all() and torch.isfinite(whole.float()).all()


@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_integer_arguments(B, call):
    """Windows, lengths and partitions are integers (Python's or NumPy's): nothing is cut
    to one or read from a text."""
    c = Case([40, 70], [1, 1], 4, 2, 64, 16, torch.float16, False, 9, 2, poison=False)
    if call == "decode":
        args = [c.max_ctx, c.window, c.sinks, 0]
        run = lambda m, w, n, P: B.pa_decode_attention_window(  # noqa: E731
            c.out, c.q, c.kc, c.vc, c.d_tables, c.d_ctx, m, c.scale, w, n, P, error_word=c.err)
    else:
        args = [c.max_ctx, c.window, c.sinks]
        run = lambda m, w, n: B.pa_prefill_attention_window(  # noqa: E731
            c.out, c.q, c.kc, c.vc, c.d_tables, c.d_start, c.d_ctx, m, c.scale, w, n,
            error_word=c.err)
    for k, good in enumerate(args):
        for bad in (good + 0.7, float(good), str(good), None, np.float64(good)):
            with pytest.raises(TypeError):
                run(*args[:k], bad, *args[k + 1:])
    assert bool((c.out == 7).all())
    run(*[t(a) for t, a in zip((np.int64, np.uint16, torch.tensor, np.int8), args)])
    c.check()


@pytest.mark.parametrize("dtype,fp8", FLOATS, ids=IDS[:2])
@pytest.mark.parametrize("span", [(0, 144), (144, 288)])
def test_decode_values_of_keys_without_weight(B, dtype, fp8, span):
    """A weight of 0 times an infinite or NaN value is not a number, in whichever
    partition it comes."""
    c = Case([288, 30, 288], [1] * 3, 8, 2, 128, 16, dtype, fp8, 5000, 0, seed=7)
    c.q[..., 1] = c.q[..., 1].abs() + 0.5
    put(c, c.kc, 0, range(*span), 1, float("-inf"))
    put(c, c.vc, 0, [span[0] + 70], 3, float("nan"))
    put(c, c.vc, 0, [span[0] + 100], 5, float("inf"))
    for P in PARTITIONS:
        c.out.fill_(7.0)
        c.decode(B, P)
        want = check(c, f"P={P}")
    assert (np.isnan(want[0]).all(0).nonzero()[0] == [3, 5]).all()


@pytest.mark.parametrize("dtype,fp8", TYPES, ids=IDS)
@pytest.mark.parametrize("P", [0, 16])
def test_decode_of_eleven_thousand_sequences(B, dtype, fp8, P):
    S = 11000
    ctx = np.random.default_rng(2).integers(1, 60, size=S)
    c = Case(ctx, [1] * S, 2, 1, 64, 16, dtype, fp8, 20, 3, seed=2)
    c.decode(B, P)
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_special_values_in_more_units_than_masks(B, fp8):
    """Sequences of more rows than tokens, 65 units a CTA and more, a NaN value at
    position 5 of each: rows before the first position are zero, rows 0 to 4 numbers, and
    later ones NaN in that element alone."""
    S, H, D, bs, rows, ctx = 5000, 4, 64, 16, 40, 20
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty((S * rows, H, D), dtype=torch.float16, device="cuda").normal_(generator=g)
    kc, vc = (torch.empty((2 * S, bs, 1, D), device="cuda").normal_(generator=g)
              for _ in range(2))
    kc, vc = (x.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.half() for x in (kc, vc))
    vc[::2, 5, 0, 9] = 0x7F if fp8 else float("nan")
    i = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    out, err = torch.full_like(q, 7), i([0])
    B.pa_prefill_attention_window(out, q, kc, vc, i(np.arange(2 * S).reshape(S, 2)),
                                  i(np.arange(S + 1) * rows), i([ctx] * S), ctx, 0.125, 100, 0,
                                  error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    x = out.view(S, rows, H, D)
    assert (x[:, :rows - ctx] == 0).all()
    nan = torch.zeros_like(x[:, rows - ctx:], dtype=torch.bool)
    nan[:, 5:, :, 9] = True
    assert torch.equal(torch.isnan(x[:, rows - ctx:]), nan)
    # row 0 sees its own key alone
    v = vc[::2, 0, 0].view(torch.float8_e4m3fn).half() if fp8 else vc[::2, 0, 0]
    assert torch.equal(x[:, rows - ctx], v[:, None].expand(S, H, D))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_and_chunk_at_once(B, fp8):
    """Windowed decode and prefill on two streams at the same time, one of them a replayed
    graph, each with a workspace of its own."""
    d = Case([3000, 700, 5, 1400], [1] * 4, 8, 2, 128, 16, torch.bfloat16, fp8, 600, 20)
    c = Case([900, 100, 641, 300] * 4, [90, 100, 64, 77] * 4, 32, 8, 64, 16, torch.bfloat16, fp8,
             90, 5)
    n = B.pa_window_workspace_bytes(4, 8, 2, 128, 3000, 600, 20, 16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    d.decode(B, 16, ws)
    c.chunk(B)
    torch.cuda.synchronize()
    want = d.out.clone(), c.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            c.chunk(B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        g.replay()
        for P in (16, 80, 16):
            d.decode(B, P, ws, stream=side)
    torch.cuda.synchronize()
    assert int(d.err.item()) == 0 and int(c.err.item()) == 0
    assert torch.equal(d.out, want[0]) and torch.equal(c.out, want[1])
