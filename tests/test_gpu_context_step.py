"""Long-context serving steps run together, as an engine runs them: step maps, rotary
cache write, block bounds, selection and attention over what was selected; or decode with
accumulated weights, an eviction and the moves it asks for.  Every index comes from
the device and each part is a replay of a captured graph."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import context_refs as C  # noqa: E402
import operator_refs as R  # noqa: E402

SCALE = 0.02


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_96_gb300 import binding
    return binding


class Engine:
    """Four requests over one pool; `ROWS` tokens at most a step."""

    S, BS, MB, ROWS, TOP = 4, 16, 20, 128, 5
    LIMIT, BUDGET, SINKS, RECENT = 150, 100, 3, 20

    def __init__(self, B, dtype, fp8, H, K, D):
        self.B, self.dtype, self.fp8, self.H, self.K, self.D = B, dtype, fp8, H, K, D
        self.kv = SCALE if fp8 else 1.0
        i = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32,  # noqa: E731
                                              device="cuda")
        S, N, T = self.S, self.S * self.MB + 3, self.ROWS
        self.N, self.max_ctx = N, self.MB * self.BS
        self.tables, self.ctx, self.new = i(S, self.MB, fill=-7), i(S), i(S)
        self.gone, self.weighted = i(S), i(S)        # evicted tokens; tokens with a weight
        order = np.random.default_rng(3).permutation(N).astype(np.int32)
        self.free, self.count = torch.as_tensor(order).cuda(), i(1, fill=N)
        self.start, self.err = i(S + 1), i(1)
        self.maps = {n: (i(n), i(n), i(n)) for n in (T, S)}
        pool = torch.uint8 if fp8 else dtype
        self.kc = torch.full((N, self.BS, K, D), 0x7F if fp8 else float("nan"), dtype=pool,
                             device="cuda")
        self.vc = self.kc.clone()
        self.codes = torch.zeros((N, K, 2, D), dtype=torch.int8, device="cuda")
        self.scales = torch.full((N, K), float("nan"), device="cuda")
        self.weights = torch.full((N, self.BS), float("nan"), device="cuda")
        self.moves = i(S, min(self.BUDGET, self.max_ctx - self.BUDGET), 2)
        self.chosen = i(T, K, self.TOP)
        self.qkv = torch.zeros((T, H + 2 * K, D), dtype=dtype, device="cuda")
        self.q, self.out = (torch.zeros((T, H, D), dtype=dtype, device="cuda") for _ in range(2))
        h = D // 2
        self.freq = torch.as_tensor((10000.0 ** (-np.arange(h) / h)).astype(np.float32)).cuda()
        n = max(B.pa_weights_workspace_bytes(S, H, K, D, self.max_ctx, 64),
                B.pa_sparse_workspace_bytes(T, H, K, D, self.TOP, self.BS, 32))
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def write(self, n):
        """Maps and cache write of the step's tokens; a token's rotary position counts
        the evicted ones before it."""
        seq, pos, slot = self.maps[n]
        B, H, K = self.B, self.H, self.K
        B.pa_build_step_maps(self.tables, self.ctx, self.new, self.free, self.count, self.BS,
                             self.N, self.start, seq, pos, slot, self.ctx, self.count,
                             error_word=self.err)
        place = pos + self.gone[seq.clamp(min=0)]
        q, k, v = (x[:n] for x in self.qkv.split([H, K, K], dim=1))
        B.pa_rope_and_cache(self.q[:n], q, k, v, self.kc, self.vc, slot, place, self.freq,
                            k_scale=self.kv, v_scale=self.kv, error_word=self.err)

    def sparse_step(self):
        """A mixed batch whose rows attend the blocks that they select."""
        n, B = self.ROWS, self.B
        seq, pos, _ = self.maps[n]
        self.write(n)
        B.pa_summarize_blocks(self.codes, self.scales, self.kc, self.tables, self.ctx, self.start,
                              error_word=self.err)
        B.pa_select_blocks(self.chosen, self.q, self.codes, self.scales, self.tables, seq, pos,
                           self.max_ctx, self.BS, 1, 2, error_word=self.err)
        B.pa_decode_attention_sparse(self.out, self.q, self.kc, self.vc, self.tables, seq, pos,
                                     self.chosen, self.D ** -0.5, 32, self.ws, self.kv, self.kv,
                                     error_word=self.err)

    def weights_step(self):
        """A decode step that adds up its weights."""
        S = self.S
        self.write(S)
        self.B.pa_decode_attention_weights(self.out[:S], self.weights, self.q[:S], self.kc,
                                           self.vc, self.weights, self.tables, self.ctx,
                                           self.weighted, self.max_ctx, self.D ** -0.5, self.ws,
                                           64, self.kv, self.kv, error_word=self.err)
        self.weighted.copy_(self.ctx)

    def evict(self):
        B = self.B
        self.gone += self.ctx
        B.pa_plan_eviction(self.moves, self.ctx, self.count, self.weights, self.tables, self.ctx,
                           self.weights, self.free, self.count, self.max_ctx, self.LIMIT,
                           self.BUDGET, self.SINKS, self.RECENT, error_word=self.err)
        self.gone -= self.ctx
        self.weighted.copy_(self.ctx)
        B.pa_move_tokens(self.kc, self.vc, self.moves, error_word=self.err)
        B.pa_summarize_blocks(self.codes, self.scales, self.kc, self.tables, self.ctx,
                              error_word=self.err)

    def values(self):
        return [C.pool_values(x, self.kv) for x in (self.kc, self.vc)]

    def host(self, *names):
        return [getattr(self, n).cpu().numpy().copy() for n in names]


def check_bounds(e):
    """Every block of every context has the bounds of its keys."""
    tables, ctx, codes, scales = e.host("tables", "ctx", "codes", "scales")
    want = codes.copy() * 0, scales.copy() * 0
    C.summarize(*want, C.values(e.kc), tables, ctx)
    for s, c in enumerate(ctx):
        at = tables[s, :-(-c // e.BS)]
        assert np.array_equal(codes[at], want[0][at]) and np.array_equal(scales[at], want[1][at])


STEPS = [("sparse", [60, 5, 0, 40]), ("weights", [1, 1, 1, 1]), ("sparse", [70, 33, 1, 24]),
         ("sparse", [1, 90, 2, 33]), ("weights", [1, 1, 1, 1]), ("weights", [1, 1, 1, 1]),
         ("sparse", [30, 22, 1, 75]), ("weights", [1, 1, 1, 1]), ("sparse", [1, 1, 120, 1]),
         ("weights", [-1, 1, 1, 1]), ("sparse", [100, 1, 27, 0]), ("weights", [1, 1, 1, 1]),
         ("weights", [1, 1, 1, 1])]


@pytest.mark.parametrize("dtype,fp8,H,K,D", [
    (torch.bfloat16, False, 8, 2, 128), (torch.float16, False, 6, 2, 64),
    (torch.bfloat16, True, 16, 1, 64), (torch.float16, True, 4, 4, 128)],
    ids=["bf16", "f16", "bf16-fp8", "f16-fp8"])
def test_steps_with_selection_and_eviction(B, dtype, fp8, H, K, D):
    e = Engine(B, dtype, fp8, H, K, D)
    graphs = {}
    state = torch.cuda.Stream()
    with torch.cuda.stream(state):
        for name in ("sparse_step", "weights_step", "evict"):
            getattr(e, name)()                       # nobody has a token yet
        torch.cuda.synchronize()
        for name in ("sparse_step", "weights_step", "evict"):
            graphs[name] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[name], stream=state):
                getattr(e, name)()
    torch.cuda.synchronize()
    p_dtype = torch.float16 if fp8 else dtype
    scale, evicted = D ** -0.5, 0
    for k, (kind, new) in enumerate(STEPS):
        what = f"step {k}"
        e.new.copy_(torch.as_tensor(new))
        e.qkv.copy_(torch.randn(e.qkv.shape, generator=torch.Generator().manual_seed(k)))
        e.out.fill_(7.0)
        before = dict(zip(("tables", "ctx", "free", "weights", "weighted"),
                          e.host("tables", "ctx", "free", "weights", "weighted")))
        gone_before = e.gone.cpu().numpy().copy()
        n = e.ROWS if kind == "sparse" else e.S
        maps = R.step_maps(before["tables"], before["ctx"], new, before["free"],
                           int(e.count.item()), e.BS, n)
        graphs[kind + "_step"].replay()
        torch.cuda.synchronize()
        assert int(e.err.item()) == 0, what
        seq, pos, slot = (x.cpu().numpy() for x in e.maps[n])
        assert np.array_equal(seq, maps["seq"]) and np.array_equal(slot, maps["slot"])
        kc, vc = e.values()
        rows = int(maps["start"][-1])
        place = pos[:rows] + gone_before[seq[:rows]]
        y, err = R.rope(e.q[:0].new_tensor(0) if rows == 0 else
                        e.qkv[:rows, :H], place[None], e.freq, np.zeros(D // 2, int), False) \
            if rows else (np.zeros((0, H, D)), 0)
        R.assert_within(e.q[:rows], y, R.HALF_STEP[dtype] * (np.abs(y) + err) + err + 1e-7, what)
        if kind == "sparse":
            check_bounds(e)
            codes, scales = e.host("codes", "scales")
            chosen = e.chosen.cpu().numpy()
            want = C.select(e.q.float().cpu().numpy(), codes, scales, maps["tables"], seq, pos,
                            e.BS, e.TOP, 1, 2, K)
            assert np.array_equal(chosen, want), what
            x, tol = C.sparse_attention(e.q, kc, vc, maps["tables"], seq, pos, chosen, scale,
                                        dtype, p_dtype)
            R.assert_within(e.out, x, tol, what)
            assert not e.out[rows:].any()
            continue
        # (a finished request's slots are the next one's: its weights start anew)
        old = np.where(np.isnan(before["weights"]), 0, before["weights"])
        x, tol, w, w_tol = C.weights_attention(e.q[:e.S], kc, vc, old, maps["tables"],
                                               maps["ctx"], before["weighted"], scale, dtype,
                                               p_dtype)
        R.assert_within(e.out[:e.S], x, tol, what)
        got = e.weights.cpu().numpy()
        for s, c in enumerate(maps["ctx"]):
            p = np.arange(c)
            at = maps["tables"][s][p // e.BS], p % e.BS
            assert (np.abs(got[at] - w[at]) <= w_tol[at]).all(), what
        # ---- the eviction --------------------------------------------------------------
        pools = [x.clone() for x in (e.kc, e.vc)]
        tables, ctx, free, weights = e.host("tables", "ctx", "free", "weights")
        want = C.plan_eviction(tables, ctx, weights, free, int(e.count.item()), e.BS, e.LIMIT,
                               e.BUDGET, e.SINKS, e.RECENT, e.moves.shape[1])
        graphs["evict"].replay()
        torch.cuda.synchronize()
        assert int(e.err.item()) == 0, what
        assert np.array_equal(e.moves.cpu().numpy(), want[0]), what
        assert np.array_equal(e.ctx.cpu().numpy(), want[1])
        assert np.array_equal(e.free.cpu().numpy(), want[2]) and int(e.count.item()) == want[3]
        assert np.array_equal(e.gone.cpu().numpy() - gone_before, ctx - want[1])
        m = want[0][want[0][..., 1] >= 0]
        evicted += len(m)
        for was, now in zip(pools, (e.kc, e.vc)):
            flat = was.view(torch.uint8).view(e.N * e.BS, -1)
            flat[torch.as_tensor(m[:, 1]).long().cuda()] = \
                flat[torch.as_tensor(m[:, 0]).long().cuda()]
            assert torch.equal(flat, now.view(torch.uint8).view(e.N * e.BS, -1)), what
        check_bounds(e)
    assert evicted > 50
