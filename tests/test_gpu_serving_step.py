"""Step maps, rotary cache write and windowed attention run together, as an
engine runs them: every step's indices come from the device, each step is a
replay of a captured graph, and the outputs are held to the definition in 64 bits.
Then the operators at offsets past 32 bits."""
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


class Engine:
    """Five requests over one small pool; `rows` tokens at most a step."""

    S, BS, MB, ROWS = 5, 16, 16, 96

    def __init__(self, B, dtype, fp8, H, K, D, window, sinks, spare):
        self.B, self.dtype, self.fp8, self.H, self.K, self.D = B, dtype, fp8, H, K, D
        self.window, self.sinks, self.kv = window, sinks, SCALE if fp8 else 1.0
        i = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32,  # noqa: E731
                                              device="cuda")
        S, N = self.S, self.S * self.MB + spare
        self.N = N
        self.tables, self.ctx, self.new = i(S, self.MB, fill=-7), i(S), i(S)
        order = np.random.default_rng(3).permutation(N).astype(np.int32)
        self.free, self.count = torch.as_tensor(order).cuda(), i(1, fill=N)
        self.start, self.err = i(S + 1), i(1)
        self.maps = {n: (i(n), i(n), i(n)) for n in (self.ROWS, S)}   # seq, pos, slot
        pool = torch.uint8 if fp8 else dtype
        self.kc = torch.full((N, self.BS, K, D), 0x7F if fp8 else float("nan"), dtype=pool,
                             device="cuda")
        self.vc = self.kc.clone()
        self.qkv = torch.zeros((self.ROWS, H + 2 * K, D), dtype=dtype, device="cuda")
        self.q = torch.zeros((self.ROWS, H, D), dtype=dtype, device="cuda")
        self.out = torch.zeros((self.ROWS, H, D), dtype=dtype, device="cuda")
        h = D // 2
        self.freq = torch.as_tensor((10000.0 ** (-np.arange(h) / h)).astype(np.float32)).cuda()
        self.max_ctx = self.MB * self.BS
        self.ws = torch.zeros(max(256, B.pa_window_workspace_bytes(S, H, K, D, self.max_ctx,
                                                                   window, sinks, 16)),
                              dtype=torch.uint8, device="cuda")
        # the same state by the definition
        self.state = dict(tables=self.tables.cpu().numpy(), free=order.copy(),
                          ctx=np.zeros(S, int), count=N)

    def step(self, n):
        """The step's four calls over n rows: windowed decode where every request
        has one, the mixed batch otherwise."""
        B, H, K = self.B, self.H, self.K
        seq, pos, slot = self.maps[n]
        B.pa_build_step_maps(self.tables, self.ctx, self.new, self.free, self.count, self.BS,
                             self.N, self.start, seq, pos, slot, self.ctx, self.count,
                             error_word=self.err)
        q, k, v = (x[:n] for x in self.qkv.split([H, K, K], dim=1))
        scales = dict(k_scale=self.kv, v_scale=self.kv, error_word=self.err)
        B.pa_rope_and_cache(self.q[:n], q, k, v, self.kc, self.vc, slot, pos, self.freq, **scales)
        head = (self.out[:n], self.q[:n], self.kc, self.vc, self.tables)
        tail = (self.ctx, self.max_ctx, self.D ** -0.5, self.window, self.sinks)
        if n == self.S:
            B.pa_decode_attention_window(*head, *tail, 16, self.ws, **scales)
        else:
            B.pa_prefill_attention_window(*head, self.start, *tail, **scales)

    def check(self, n, new, what):
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0, what
        was = self.state
        want = R.step_maps(was["tables"], was["ctx"], new, was["free"], was["count"], self.BS, n)
        self.state = want
        seq, pos, slot = (x.cpu().numpy() for x in self.maps[n])
        for name, a in dict(start=self.start, ctx=self.ctx, tables=self.tables,
                            free=self.free).items():
            assert np.array_equal(a.cpu().numpy(), want[name]), (what, name)
        assert int(self.count.item()) == want["count"]
        for name, a in dict(seq=seq, pos=pos, slot=slot).items():
            assert np.array_equal(a, want[name]), (what, name)
        rows = int(want["start"][-1])
        qkv = self.qkv[:rows]
        q, k, v = qkv.split([self.H, self.K, self.K], dim=1)
        half, live = R.HALF_STEP[self.dtype], pos[None, :rows]
        axis = np.zeros(self.D // 2, int)
        y, e = R.rope(q, live, self.freq, axis, False)
        R.assert_within(self.q[:rows], y, half * (np.abs(y) + e) + e + 1e-7, what)
        y, e = R.rope(k, live, self.freq, axis, False)
        kc, vc = (R.pool_values(x, self.kv) for x in (self.kc, self.vc))
        flat = kc.reshape(-1, self.K, self.D)[slot[:rows]]
        if self.fp8:
            tol = np.maximum(np.abs(y) * 2.0 ** -4, SCALE * 2.0 ** -10) + e * 1.07 + 1e-6
        else:
            tol = half * (np.abs(y) + e) + e + 1e-7
        assert (np.abs(flat - y) <= tol).all(), what
        x, tol = R.window_attention(self.q[:rows], kc, vc, want["tables"], want["start"],
                                    want["ctx"], self.D ** -0.5, self.window, self.sinks,
                                    self.dtype, torch.float16 if self.fp8 else self.dtype)
        R.assert_within(self.out[:rows], x, tol, what)
        # rows past the step's are left as they were
        assert bool((self.out[rows:n] == 7).all()), what


# tokens per request and step; -1: the request ends and its blocks go to others
STEPS = [[37, 5, 16, 1, 0], [1, 40, 1, 33, 20], [1, 1, 1, 1, 1], [1, 1, 1, 1, 1],
         [-1, 50, 1, 1, 1], [64, 1, 1, -1, 1], [1, 1, 17, 16, 1], [1, 1, 1, 1, 1],
         [1, 1, -1, 1, 60], [1, 1, 31, 1, 1], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0],
         [1, 1, 1, 1, 1], [-1, -1, -1, -1, -1], [2, 0, 3, 0, 90], [1, 1, 1, 1, 1]]


@pytest.mark.parametrize("dtype,fp8,H,K,D,window,sinks", [
    (torch.bfloat16, False, 8, 2, 128, 24, 4), (torch.float16, False, 6, 2, 64, 17, 0),
    (torch.bfloat16, True, 8, 1, 128, 40, 17), (torch.float16, True, 4, 4, 64, 1000, 4)])
def test_replayed_steps(B, dtype, fp8, H, K, D, window, sinks):
    e = Engine(B, dtype, fp8, H, K, D, window, sinks, spare=2)
    graphs = {}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):      # (nothing to do: every request brings no token)
        for n in (e.ROWS, e.S):
            e.step(n)
    torch.cuda.synchronize()
    for n in (e.ROWS, e.S):         # both graphs use one state, one pool and one workspace
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            e.step(n)
    gen = torch.Generator().manual_seed(11)
    for i, new in enumerate(STEPS):
        n = e.S if all(x == 1 for x in new) else e.ROWS
        e.new.copy_(torch.as_tensor(new, dtype=torch.int32))
        e.qkv.copy_(torch.randn(e.qkv.shape, generator=gen))
        e.out.fill_(7)
        graphs[n].replay()
        e.check(n, new, f"step {i}")


@pytest.mark.parametrize("fp8", [False, True])
def test_pools_past_32_bits(B, fp8):
    """Blocks whose rows start past 2^32 bytes (2^32 elements of FP8 pools)."""
    K, D, bs, dtype = 8, 128, 256, torch.bfloat16
    need = torch.cuda.mem_get_info()[0]
    N = (1 << 32) // (bs * K * D * (1 if fp8 else 2)) + 6
    if need < 12 << 30:
        pytest.skip("12 GB of device memory")
    kc, vc = (torch.empty((N, bs, K, D), dtype=torch.uint8 if fp8 else dtype, device="cuda")
              for _ in range(2))
    T = 300
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((T, h, D), generator=gen).to(dtype).cuda() for h in (16, K, K))
    table = torch.tensor([[N - 1, N - 3]], dtype=torch.int32).cuda()
    i = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    slots = [(N - 1) * bs + p if p < bs else (N - 3) * bs + p - bs for p in range(T)]
    freq = torch.zeros(D // 2, device="cuda")
    err = i([0])
    kv = SCALE if fp8 else 1.0
    kw = dict(k_scale=kv, v_scale=kv, error_word=err)
    out = torch.empty_like(q)
    B.pa_rope_and_cache(out, q, k, v, kc, vc, i(slots), i(range(T)), freq, **kw)
    assert torch.equal(out, q)
    small = [R.pool_values(x[N - 3:], kv) for x in (kc, vc)]
    want_k = k.double().cpu().numpy()
    got_k = np.concatenate([small[0][2], small[0][0]])[:T]
    if fp8:
        assert (np.abs(got_k - want_k) <= np.maximum(np.abs(want_k) * 2.0 ** -4,
                                                     SCALE * 2.0 ** -10) + 1e-6).all()
    else:
        assert np.array_equal(got_k, want_k)
    scale, window, sinks = D ** -0.5, 70, 5
    B.pa_prefill_attention_window(out, q, kc, vc, table, i([0, T]), i([T]), T, scale, window,
                                  sinks, **kw)
    tables = np.array([[2, 0]])
    p_dtype = torch.float16 if fp8 else dtype
    want, tol = R.window_attention(q, *small, tables, [0, T], [T], scale, window, sinks, dtype,
                                   p_dtype)
    R.assert_within(out, want, tol, "chunk")
    one = torch.empty_like(q[:1])
    B.pa_decode_attention_window(one, q[T - 1:], kc, vc, table, i([T]), T, scale, window, sinks,
                                 0, None, **kw)
    R.assert_within(one, want[T - 1:], tol[T - 1:], "decode")
    assert int(err.item()) == 0


def test_rows_past_32_bits(B):
    """Query rows past 2^31 elements of a long chunk and of a long rotary batch."""
    H, K, D, bs, dtype = 64, 4, 128, 64, torch.bfloat16
    T = (1 << 31) // (H * D) + 70
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("24 GB of device memory")
    MB = -(-T // bs)
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.empty((T, H, D), dtype=dtype, device="cuda").normal_(generator=gen)
    k, v = (torch.empty((T, K, D), dtype=dtype, device="cuda").normal_(generator=gen)
            for _ in range(2))
    kc, vc = (torch.empty((MB, bs, K, D), dtype=dtype, device="cuda") for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = torch.as_tensor((10000.0 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    B.pa_rope_and_cache(out, q, k, v, kc, vc, pos, pos, freq, error_word=err)
    last = 40
    y, e = R.rope(q[-last:], pos[None, -last:].cpu().numpy(), freq, np.zeros(64, int), False)
    R.assert_within(out[-last:], y, 2.0 ** -8 * (np.abs(y) + e) + e + 1e-7, "rope")
    q, out = out, q
    window, sinks = 16, 3
    table = torch.arange(MB, dtype=torch.int32, device="cuda")[None]
    i = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    B.pa_prefill_attention_window(out, q, kc, vc, table, i([0, T]), i([T]), T, D ** -0.5, window,
                                  sinks, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, tol = R.window_attention(q[-last:], R.pool_values(kc), R.pool_values(vc),
                                   table.cpu().numpy(), [0, last], [T], D ** -0.5, window, sinks,
                                   dtype, dtype)
    R.assert_within(out[-last:], want, tol, "chunk")


@pytest.mark.parametrize("fp8", [False, True])
def test_as_many_sequences_as_a_launch_takes(B, fp8):
    S, H, K, D, bs, dtype = 5120, 2, 1, 64, 16, torch.float16
    rng = np.random.default_rng(1)
    rows = rng.integers(0, 3, size=S)
    ctx = rows + rng.integers(0, 30, size=S)
    start = np.concatenate([[0], np.cumsum(rows)])
    T, MB = int(start[-1]), 2
    gen = torch.Generator().manual_seed(5)
    q = torch.randn((T, H, D), generator=gen).to(dtype).cuda()
    k, v = (torch.randn((64, bs, K, D), generator=gen).to(dtype) for _ in range(2))
    if fp8:
        k, v = (x.float().to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    kc, vc = k.cuda(), v.cuda()
    tables = rng.integers(0, 64, size=(S, MB)).astype(np.int32)
    i = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    out = torch.full_like(q, 7)
    err = i([0])
    B.pa_prefill_attention_window(out, q, kc, vc, i(tables), i(start), i(ctx), 32, 0.125, 9, 2,
                                  error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, tol = R.window_attention(q, R.pool_values(kc), R.pool_values(vc), tables, start, ctx,
                                   0.125, 9, 2, dtype, dtype)
    R.assert_within(out, want, tol)
