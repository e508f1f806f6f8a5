"""pa_rope_and_cache against the rotation in 64 bits, and its cache write
against the pools' own rules."""
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


SCALE = 0.0137


def make(T, H, K, D, rot, dtype, fp8, axes, max_pos, fused, seed, bs=16):
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    qkv = torch.randn((T, H + 2 * K, D), generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    N = T // bs + 3
    pool = torch.uint8 if fp8 else dtype
    kc = torch.full((N, bs, K, D), 0x5A if fp8 else float("nan"), dtype=pool, device="cuda")
    vc = kc.clone()
    slots = r.permutation(N * bs)[:T].astype(np.int32)
    pos = r.integers(0, max_pos, size=(axes, T)).astype(np.int32)
    h = rot // 2
    freq = torch.as_tensor((10000.0 ** (-2.0 * np.arange(h) / rot)).astype(np.float32))
    axis = torch.as_tensor((np.arange(h) * 3 // h % axes).astype(np.int32))
    return dict(q=q, k=k, v=v, kc=kc, vc=vc, slots=torch.as_tensor(slots).cuda(),
                pos=torch.as_tensor(pos).cuda(), freq=freq.cuda(), axis=axis, qkv=qkv)


def call(B, s, out, **kw):
    B.pa_rope_and_cache(out, s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"],
                        s["freq"], axis_of_pair=s["axis"], **kw)


def check(s, out, q, k, v, kc0, dtype, fp8, interleaved):
    pos, axis = s["pos"].cpu().numpy().reshape(-1, q.shape[0]), s["axis"].numpy()
    want, err = R.rope(q, pos, s["freq"], axis, interleaved)
    half = R.HALF_STEP[dtype]
    R.assert_within(out, want, half * (np.abs(want) + err) + err + 1e-7, "query")
    kr, kerr = R.rope(k, pos, s["freq"], axis, interleaved)
    slots = s["slots"].cpu().numpy()
    live = np.flatnonzero(slots >= 0)
    flat = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
    kc, vc = flat(s["kc"]), flat(s["vc"])
    at = torch.as_tensor(slots[live].astype(np.int64)).cuda()
    if fp8:
        inv = float(np.float32(1) / np.float32(SCALE))
        x = np.clip(kr[live] * inv, -448, 448)
        # half a step of e4m3: 2^-4 of the value, 2^-10 below the normal range
        tol = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10) + kerr[live] * inv * 1.07 + 1e-5
        R.assert_within(kc[at].view(torch.float8_e4m3fn).float(), x, tol, "key codes")
        vx = (v.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(vc[at], vx[live])
    else:
        R.assert_within(kc[at], kr[live], half * (np.abs(kr) + kerr)[live] + kerr[live] + 1e-7,
                        "key")
        assert torch.equal(vc[at], v[live])
    # every other slot is left as it was
    other = torch.ones(kc.shape[0], dtype=torch.bool, device="cuda")
    other[at] = False
    raw = torch.uint8 if fp8 else torch.int16
    for c in (kc, vc):
        assert torch.equal(c[other].view(raw), flat(kc0)[other].view(raw))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,K,D,rot,axes,interleaved,fused,max_pos", [
    (1, 1, 1, 64, 64, 1, False, True, 10),
    (4, 4, 4, 64, 64, 1, False, True, 4096),
    (5, 6, 2, 64, 32, 1, True, False, 1000),
    (37, 64, 8, 128, 128, 3, False, True, 1000000),
    (130, 8, 1, 128, 64, 3, False, True, 131072),
    (19, 5, 5, 128, 128, 2, True, True, 2 ** 31 - 1),
    (7, 3, 1, 256, 256, 1, False, False, 2 ** 24),
    (3, 2, 1, 16, 16, 1, True, True, 100),
    (300, 40, 8, 48, 16, 2, False, True, 50000),
    (2, 128, 16, 128, 112, 3, False, False, 300),
    # long batches: units of one token and of parts of a token
    (2101, 100, 14, 128, 128, 3, False, True, 131072),
    (2101, 96, 16, 128, 96, 2, True, True, 131072),
    (1401, 80, 8, 256, 192, 1, False, False, 2 ** 20),
    (16001, 16, 1, 128, 128, 1, False, True, 2 ** 31 - 1),
    (16011, 40, 2, 48, 16, 2, True, False, 1000)])
def test_matches_the_definition(B, fp8, dtype, T, H, K, D, rot, axes, interleaved, fused, max_pos):
    s = make(T, H, K, D, rot, dtype, fp8, axes, max_pos, fused, T * 7 + D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if T > 3:
        s["slots"][T // 2] = -1   # padding: rotated, not cached
    out = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda")
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    call(B, s, out, interleaved=interleaved, k_scale=SCALE, v_scale=SCALE, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(s, out, q, k, v, kc0, dtype, fp8, interleaved)
    assert torch.equal(s["q"], q) and torch.equal(s["k"], k) and torch.equal(s["v"], v)


@pytest.mark.parametrize("fp8", [False, True])
def test_in_place_inside_the_fused_rows(B, fp8):
    """The rotated query over the query's own part of the QKV rows, whose other
    parts are left as they are."""
    dtype = torch.bfloat16
    s = make(65, 16, 2, 128, 128, dtype, fp8, 3, 9000, True, 3)
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    call(B, s, s["q"], k_scale=SCALE, v_scale=SCALE)
    torch.cuda.synchronize()
    check(s, s["q"], q, k, v, kc0, dtype, fp8, False)
    assert torch.equal(s["k"], k) and torch.equal(s["v"], v)


def test_output_between_other_parts_of_a_row(B):
    """Input and output rows side by side in wider rows."""
    T, H, K, D = 33, 4, 2, 64
    wide = torch.randn((T, 2 * H + 2 * K, D)).half().cuda()
    s = make(T, H, K, D, D, torch.float16, False, 1, 100, True, 9)
    s["q"], s["k"], s["v"] = wide[:, :H], wide[:, 2 * H:2 * H + K], wide[:, 2 * H + K:]
    out = wide[:, H:2 * H]
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    call(B, s, out)
    torch.cuda.synchronize()
    check(s, out, q, k, v, kc0, torch.float16, False, False)
    with pytest.raises(B.PAError):
        call(B, s, wide[:, H - 1:2 * H - 1])  # half over the query's rows


def test_equals_the_cache_write_where_nothing_turns(B):
    """Position 0 turns nothing: pools bit for bit those of pa_reshape_and_cache."""
    for fp8 in (False, True):
        s = make(50, 8, 2, 128, 128, torch.bfloat16, fp8, 1, 5, False, 11)
        s["pos"].zero_()
        kc, vc = s["kc"].clone(), s["vc"].clone()
        out = torch.empty_like(s["q"])
        call(B, s, out, k_scale=SCALE, v_scale=SCALE)
        if fp8:
            B.pa_reshape_and_cache_fp8(s["k"], s["v"], kc, vc, s["slots"], SCALE, SCALE)
        else:
            B.pa_reshape_and_cache(s["k"], s["v"], kc, vc, s["slots"])
        torch.cuda.synchronize()
        raw = torch.uint8 if fp8 else torch.int16
        assert torch.equal(s["kc"].view(raw), kc.view(raw))
        assert torch.equal(s["vc"].view(raw), vc.view(raw))
        assert torch.equal(out, s["q"])


def test_bad_slots_are_skipped_and_flagged(B):
    s = make(20, 4, 2, 64, 64, torch.bfloat16, False, 1, 50, True, 12)
    N = s["kc"].shape[0] * s["kc"].shape[1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["slots"][3], s["slots"][9], s["slots"][19] = N, 2 ** 31 - 1, -5
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    out = torch.empty_like(q)
    call(B, s, out, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.DEVERR_SLOT_RANGE
    s["slots"][3] = s["slots"][9] = -1
    check(s, out, q, k, v, kc0, torch.bfloat16, False, False)


def test_negative_positions_and_special_values(B):
    """A negative position turns the other way; NaN and infinities stay in their
    own pairs."""
    s = make(8, 2, 1, 64, 64, torch.float16, False, 1, 5, False, 13)
    s["pos"].copy_(torch.tensor([[-1, -5000, -2 ** 31, 7, 0, 3, 1, 2]], dtype=torch.int32))
    s["q"][3, 0, 5] = float("nan")
    s["q"][5, 1, 40] = float("inf")
    out = torch.empty_like(s["q"])
    q, kc0 = s["q"].clone(), s["kc"].clone()
    call(B, s, out)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(out)
    where = {tuple(x) for x in torch.nonzero(bad).tolist()}
    assert where == {(3, 0, 5), (3, 0, 37), (5, 1, 8), (5, 1, 40)}
    q[3, 0, 5] = q[3, 0, 37] = q[5, 1, 8] = q[5, 1, 40] = 0
    out[bad] = 0
    check(s, out, q, s["k"], s["v"], kc0, torch.float16, False, False)


def test_captured_and_on_another_stream(B):
    s = make(40, 8, 2, 128, 128, torch.bfloat16, False, 1, 500, True, 14)
    out = torch.empty((40, 8, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(B, s, out, stream=side)
    torch.cuda.synchronize()
    check(s, out, q, k, v, kc0, torch.bfloat16, False, False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(B, s, out)
    s["pos"].add_(123456)
    s["kc"].copy_(kc0)
    s["vc"].copy_(kc0)
    g.replay()
    torch.cuda.synchronize()
    check(s, out, q, k, v, kc0, torch.bfloat16, False, False)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_batch_in_place_with_bad_slots(B, fp8):
    """In place in the fused rows; slots that are negative or past the pool
    write nothing, and only the latter are flagged."""
    s = make(2300, 100, 14, 128, 128, torch.bfloat16, fp8, 3, 131072, True, 21)
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    N, bs = s["kc"].shape[:2]
    good = s["slots"].clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(k_scale=SCALE, v_scale=SCALE) if fp8 else {}
    s["slots"][5::7] = -1
    call(B, s, s["q"], error_word=err, **kw)
    assert int(err.item()) == 0
    check(s, s["q"], q, k, v, kc0, torch.bfloat16, fp8, False)
    for name, x in dict(q=q, kc=kc0, vc=kc0).items():
        s[name].copy_(x)
    s["slots"].copy_(good)
    bad = torch.arange(3, 2300, 11, device="cuda")
    s["slots"][bad] = N * bs
    call(B, s, s["q"], error_word=err, **kw)
    assert int(err.item()) == B.DEVERR_SLOT_RANGE
    s["slots"][bad] = -1
    check(s, s["q"], q, k, v, kc0, torch.bfloat16, fp8, False)


def test_long_batch_captured_beside_another(B):
    """Two long batches on two streams at once, one of them a captured graph."""
    a, b = (make(2300, 100, 14, 128, 128, torch.bfloat16, False, 3, 131072, True, i)
            for i in (31, 32))
    outs = [torch.empty_like(x["q"].contiguous()) for x in (a, b)]
    kept = [(x["q"].clone(), x["k"].clone(), x["v"].clone(), x["kc"].clone()) for x in (a, b)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(B, a, outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        g.replay()
        call(B, b, outs[1], stream=side)
    torch.cuda.synchronize()
    for x, o, (q, k, v, kc0) in zip((a, b), outs, kept):
        check(x, o, q, k, v, kc0, torch.bfloat16, False, False)


def test_long_batch_wait_limit(B):
    """A copy that never comes ends in a flag, and the next call is whole."""
    s = make(2300, 100, 14, 128, 128, torch.bfloat16, False, 3, 131072, True, 41)
    out = torch.empty((2300, 100, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v, kc0 = s["q"].clone(), s["k"].clone(), s["v"].clone(), s["kc"].clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.pa_set_stage_wait_limit_ns(2_000_000)
    B.pa_debug_withhold_first_fill(True)
    try:
        call(B, s, out, error_word=err)
        torch.cuda.synchronize()
    finally:
        B.pa_debug_withhold_first_fill(False)
        B.pa_set_stage_wait_limit_ns(0)
    assert int(err.item()) == B.DEVERR_TIMEOUT
    err.zero_()
    call(B, s, out, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(s, out, q, k, v, kc0, torch.bfloat16, False, False)


def test_binding_checks_every_tensor(B):
    s = make(9, 4, 2, 64, 64, torch.float16, False, 1, 50, True, 51)
    out = torch.full((9, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    kept = s["kc"].clone()
    for name, bad, error in (
            ("q", s["q"].float(), TypeError), ("q", s["q"].cpu(), ValueError),
            ("q", s["q"][..., ::2], ValueError), ("q", s["q"][:, ::2], ValueError),
            ("k", s["k"].bfloat16(), TypeError), ("k", s["k"][:8], ValueError),
            ("v", s["v"].cpu(), ValueError), ("v", s["v"][:, :, ::2], ValueError),
            ("kc", s["kc"].bfloat16(), TypeError), ("vc", s["vc"][:-1], ValueError),
            ("slots", s["slots"].long(), TypeError), ("slots", s["slots"][:-1], ValueError),
            ("pos", s["pos"][:, :-1], ValueError), ("pos", s["pos"].cpu(), ValueError),
            ("pos", s["pos"][None], ValueError), ("freq", s["freq"].double(), TypeError),
            ("freq", s["freq"][None], ValueError), ("axis", s["axis"].cuda(), ValueError),
            ("axis", s["axis"][1:], ValueError), ("axis", s["axis"] + 1, B.PAError)):
        with pytest.raises(error):
            call(B, dict(s, **{name: bad}), out)
    with pytest.raises(TypeError):
        call(B, s, out, error_word=torch.zeros(1, device="cuda"))
    torch.cuda.synchronize()
    assert bool((out == 7).all())
    assert torch.equal(s["kc"].view(torch.int16), kept.view(torch.int16))
