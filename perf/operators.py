"""Measured cases of the serving-step operators around the paged KV cache.

Four operators, in the order a serving step runs them:

  maps    block tables, query offsets and slots of a step's new tokens, built
          on the GPU from each request's length and number of new tokens
          (``pa_build_step_maps``)
  rope    rotary positions with one to three axes applied to the queries and
          keys of the new tokens, keys and values written to the paged pools
          (``pa_rope_and_cache``)
  decode  paged decode attention with a sliding window and a few first tokens
          that stay visible (``pa_decode_attention_window``)
  chunk   the same window for chunks of new tokens, many rows per sequence
          (``pa_prefill_attention_window``)

Lengths are drawn from a case's own ``lens`` number, so that its work is known
from the case alone; values, block placement and positions come from the seed
of ``prepare``.  Pools hold finite values everywhere, as a pool whose blocks
were used before does.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

THETA = 10000.0
FP8_SCALE = 0.0137  # per-pool scale of e4m3 codes, N(0, 1) values


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # 128 running requests, one new token each: the metadata of a decode step
        dict(name="maps decode 128", op="maps", seqs=128, tokens=128, block=16, max_blocks=512,
             prompts=0, chunk=1, finished=0, idle=0, lens=11),
        # continuous batching: decode requests, prompt chunks within a budget
        # of 2048 tokens (the tail is padding), some requests finish or wait
        dict(name="maps mixed 61", op="maps", seqs=61, tokens=2048, block=16, max_blocks=256,
             prompts=5, chunk=512, finished=7, idle=3, lens=12),
        # a large server: thousands of requests and 64k new tokens
        dict(name="maps 4096 requests", op="maps", seqs=4096, tokens=65536, block=32,
             max_blocks=512, prompts=100, chunk=600, finished=300, idle=64, lens=13),
        # four short chats on a small model, fp16
        dict(name="rope 4 tokens d64", op="rope", tokens=4, heads=4, kv_heads=4, dim=64, rot=64,
             block=16, dtype="f16", kv="same", axes=1, interleaved=False, fused=True,
             max_pos=4096, pad=0),
        # a GQA decode step of 128 requests over an FP8 cache, far positions
        dict(name="rope decode 128 fp8", op="rope", tokens=128, heads=64, kv_heads=8, dim=128,
             rot=128, block=16, dtype="bf16", kv="fp8", axes=1, interleaved=False, fused=True,
             max_pos=1000000, pad=0),
        # prompts with images and video: time, height and width, fused QKV rows
        dict(name="rope video 16381", op="rope", tokens=16381, heads=64, kv_heads=8, dim=128,
             rot=128, block=16, dtype="bf16", kv="same", axes=3, interleaved=False, fused=True,
             max_pos=131072, pad=37),
        # four short chats, window shorter than some contexts
        dict(name="window decode 4 d64", op="decode", seqs=4, heads=4, kv_heads=4, dim=64, block=16,
             dtype="f16", kv="same", window=128, sinks=4, min_ctx=1, max_ctx=500, partition=0,
             lens=31),
        # a GQA 70B-like decode layer, 128 requests
        dict(name="window decode gqa 1024", op="decode", seqs=128, heads=64, kv_heads=8, dim=128,
             block=16, dtype="bf16", kv="same", window=1024, sinks=4, min_ctx=16, max_ctx=8192,
             partition=1024, lens=32),
        # long contexts over an FP8 cache, few requests, window split in partitions
        dict(name="window decode long fp8", op="decode", seqs=16, heads=32, kv_heads=8, dim=128,
             block=32, dtype="bf16", kv="fp8", window=4096, sinks=16, min_ctx=64, max_ctx=32768,
             partition=512, lens=33),
        # a mixed batch on a small model: decode rows and short prompts
        dict(name="window mixed 82 rows", op="chunk", seqs=4, rows=82, heads=8, kv_heads=2, dim=64,
             block=16, dtype="f16", kv="same", window=33, sinks=3, max_ctx=70, lens=41),
        # chunked prefill: a budget of 2048 tokens over four prompts
        dict(name="window chunked 2048", op="chunk", seqs=4, rows=2048, heads=64, kv_heads=8,
             dim=128, block=16, dtype="bf16", kv="same", window=512, sinks=4, max_ctx=2048,
             lens=42),
        # long prompts behind a wide window
        dict(name="window long 8192", op="chunk", seqs=4, rows=8192, heads=32, kv_heads=8, dim=128,
             block=32, dtype="bf16", kv="same", window=4096, sinks=64, max_ctx=32768, lens=43),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    """Query heads, KV heads and head size."""
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), kv, rng.choice([64, 128])


def draw(rng):
    op = rng.choice(["maps", "rope", "decode", "chunk"])
    lens = rng.randrange(1, 1 << 30)
    block = rng.choice([16, 32, 64])
    if op == "maps":
        seqs = _log(rng, 1, 4096)
        prompts = rng.randint(0, min(seqs, 64))
        chunk = _log(rng, 1, 800)
        rest = seqs - prompts
        finished = rng.randint(0, rest // 4)
        idle = rng.randint(0, rest // 8)
        tokens = rest + prompts * chunk + rng.choice([0, 0, rng.randint(1, 300)])
        return dict(op=op, seqs=seqs, tokens=min(tokens, 65536), block=block,
                    max_blocks=_log(rng, 64, 512), prompts=prompts, chunk=chunk,
                    finished=finished, idle=idle, lens=lens)
    dtype = rng.choice(["f16", "bf16"])
    kv = rng.choice(["same", "same", "fp8"])
    heads, kv_heads, dim = _heads(rng)
    if op == "rope":
        most = int(16381 * 80 * 128 / ((heads + 2 * kv_heads) * dim))
        return dict(op=op, tokens=_log(rng, 1, min(16384, most)), heads=heads, kv_heads=kv_heads,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2]), block=block, dtype=dtype, kv=kv,
                    axes=rng.randint(1, 3), interleaved=rng.random() < 0.3,
                    fused=rng.random() < 0.7, max_pos=_log(rng, 1000, 1000000),
                    pad=rng.choice([0, rng.randint(1, 50)]))
    window = _log(rng, 16, 4096)
    sinks = rng.choice([0, rng.randint(1, 128)])
    if op == "decode":
        seqs = _log(rng, 1, 256)
        room = int(128 * 1028 * 8 * 128 / (kv_heads * dim))  # tokens the largest case streams
        window = max(16, min(window, room // seqs))
        case = dict(op=op, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
                    dtype=dtype, kv=kv, window=window, sinks=sinks, min_ctx=1,
                    max_ctx=_log(rng, 64, 32768), partition=rng.choice([0, 256, 512, 1024]),
                    lens=lens)
        if case["partition"] == 0 and seqs * kv_heads < 64:
            case["partition"] = 256
        return case
    seqs = _log(rng, 1, 16)
    rows = max(seqs, _log(rng, 8, 4096))
    window = max(16, min(window, int(8192 * 32 * 4096 * 128 / (2 * rows * heads * dim))))
    return dict(op=op, seqs=seqs, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
                dtype=dtype, kv=kv, window=window, sinks=sinks,
                max_ctx=max(4 * rows // seqs + 16, _log(rng, 64, 16384)), lens=lens)


# ---------------------------------------------------------------------------
# lengths (from the case alone) and work

def _maps_lens(c):
    """Context lengths before the step and new tokens (-1: finished)."""
    r = np.random.default_rng(c["lens"])
    S, cap = c["seqs"], c["max_blocks"] * c["block"]
    new = np.ones(S, dtype=np.int64)
    who = r.permutation(S)
    p, f, i = c["prompts"], c["finished"], c["idle"]
    new[who[p:p + f]] = -1
    new[who[p + f:p + f + i]] = 0
    room = c["tokens"] - int((new[who[p:]] > 0).sum())  # tokens left for the prompts' chunks
    if p:
        new[who[:p]] = np.minimum(r.integers(1, c["chunk"] + 1, size=p), max(0, room // p))
    top = max(1, cap - int(new.max()))
    ctx = np.minimum(np.exp(r.normal(math.log(max(2, cap / 6)), 0.9, size=S)), top).astype(np.int64)
    ctx[who[:p:2]] = 0  # fresh prompts
    return ctx, new


def _decode_lens(c):
    r = np.random.default_rng(c["lens"])
    hi, lo = c["max_ctx"], min(c["min_ctx"], c["max_ctx"])
    x = np.exp(r.normal(math.log(max(lo, hi / 4)), 0.8, size=c["seqs"]))
    x = np.clip(np.rint(x), lo, hi).astype(np.int64)
    x[0] = hi
    return x


def _chunk_lens(c):
    """Context lengths (counting the chunk) and rows of each sequence."""
    r = np.random.default_rng(c["lens"])
    S, T = c["seqs"], c["rows"]
    share = r.uniform(0.5, 1.5, size=S)
    q = np.maximum(1, (share / share.sum() * (T - S)).astype(np.int64) + 1)
    q[0] += T - int(q.sum())
    if S >= 4 and T < 256:  # a mixed batch: two decode rows, the rest prompts
        q[2] += q[0] + q[1] - 2
        q[0] = q[1] = 1
    ctx = np.maximum(q, r.integers(1, max(2, c["max_ctx"] + 1), size=S))
    ctx[-1] = max(int(q[-1]), c["max_ctx"])
    return ctx, q


def _visible(pos, window, sinks):
    """Positions a query at `pos` sees."""
    n = np.asarray(pos, dtype=np.int64) + 1
    return np.minimum(n, window + np.minimum(sinks, np.maximum(0, n - window)))


def work(case):
    c = case
    if c["op"] == "maps":
        ctx, new = _maps_lens(c)
        b = c["block"]
        have = -(-ctx // b)
        taken = int((-(-(ctx + np.maximum(new, 0)) // b) - have).sum())
        given = int(have[new < 0].sum())
        # lengths in and out, offsets, 12 bytes a token, each block id moved once
        return {"bytes": 20 * c["seqs"] + 12 * c["tokens"] + 8 * taken + 8 * given, "flops": 0}
    e = 1 if c["kv"] == "fp8" else 2
    if c["op"] == "rope":
        T, D, H, K = c["tokens"], c["dim"], c["heads"], c["kv_heads"]
        return {"bytes": T * D * (2 * H * 2 + 2 * K * 2 + 2 * K * e) + 4 * T * (c["axes"] + 1),
                "flops": 3 * T * (H + K) * c["rot"]}
    D, H, K = c["dim"], c["heads"], c["kv_heads"]
    if c["op"] == "decode":
        vis = int(_visible(_decode_lens(c) - 1, c["window"], c["sinks"]).sum())
        return {"bytes": vis * K * D * 2 * e + 4 * c["seqs"] * H * D, "flops": 4 * vis * H * D}
    ctx, q = _chunk_lens(c)
    first = ctx - q
    seen = int(np.sum([_visible(np.arange(a, b), c["window"], c["sinks"]).sum()
                       for a, b in zip(first, ctx)]))
    start = np.maximum(0, first + 1 - c["window"])  # keys of the chunk's union, read once
    keys = int((ctx - start + np.minimum(c["sinks"], start)).sum())
    return {"bytes": keys * K * D * 2 * e + 4 * int(q.sum()) * H * D, "flops": 4 * seen * H * D}


# ---------------------------------------------------------------------------
# inputs

def _dev():
    return torch.device("cuda")


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).to(_dev())


def _type(c):
    return torch.float16 if c["dtype"] == "f16" else torch.bfloat16


def _tables(rng, blocks, width, spare):
    """A shuffled placement: block_tables [S, width] (unused entries 0) and
    the blocks left over."""
    total = int(blocks.sum())
    ids = rng.permutation(total + spare).astype(np.int32)
    t = np.zeros((len(blocks), width), dtype=np.int32)
    t[np.arange(width)[None, :] < blocks[:, None]] = ids[:total]
    return t, ids[total:]


def _pool(c, g, num_blocks):
    shape = (num_blocks, c["block"], c["kv_heads"], c["dim"])
    x = torch.randn(shape, generator=g, device=_dev(), dtype=torch.float32 if c["kv"] == "fp8"
                    else _type(c))
    if c["kv"] == "fp8":
        return (x / FP8_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def _prepare_maps(c, seed):
    r = np.random.default_rng(seed)
    ctx, new = _maps_lens(c)
    b = c["block"]
    have = -(-ctx // b)
    need = int((-(-(ctx + np.maximum(new, 0)) // b) - have).sum())
    t, spare = _tables(r, have, c["max_blocks"], need + 64)
    n = int(have.sum()) + need + 64
    free = np.full(n, -1, dtype=np.int32)
    free[:len(spare)] = spare
    S, T = c["seqs"], c["tokens"]
    z = lambda k: torch.zeros(k, dtype=torch.int32, device=_dev())  # noqa: E731
    return dict(op="maps", block=b, num_blocks=n, tables=_i32(t), ctx=_i32(ctx), new=_i32(new),
                free=_i32(free), count=_i32([len(spare)]), start=z(S + 1), seq=z(T), pos=z(T),
                slot=z(T), ctx_out=z(S), count_out=z(1), err=z(1))


def _positions(c, r):
    """[axes, T]: runs of text, where the axes agree, between image and video
    patches, where time, height and width run over a grid."""
    T = c["tokens"]
    at = np.sort(r.integers(0, c["max_pos"], size=T)) if T < 512 else \
        np.arange(T) + int(r.integers(0, max(1, c["max_pos"] - T)))
    i = np.arange(T)
    grid = (i // 480) % 2 == 1  # every other run of 480 tokens is 4 frames of 8 x 15 patches
    k = i % 480
    base = at - k
    p = np.stack([np.where(grid, base + k // 120, at), np.where(grid, base + k % 120 // 15, at),
                  np.where(grid, base + k % 15, at)])
    return np.maximum(p[:c["axes"]], 0)


def _prepare_rope(c, seed):
    r = np.random.default_rng(seed)
    g = torch.Generator(device=_dev()).manual_seed(int(seed))
    T, H, K, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    if c["fused"]:  # views into the rows of one projection's output
        qkv = torch.randn((T, H + 2 * K, D), generator=g, device=_dev(), dtype=_type(c))
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    else:
        q, k, v = (torch.randn((T, n, D), generator=g, device=_dev(), dtype=_type(c))
                   for n in (H, K, K))
    half = c["rot"] // 2
    n = -(-T * 5 // (4 * c["block"])) + 1
    slots = r.permutation(n * c["block"])[:T].astype(np.int32)
    if c["pad"]:
        slots[max(1, T - c["pad"]):] = -1  # padding rows at the end of the batch
    # height and width take the higher frequencies' share in thirds of the pairs
    axis = np.minimum(np.arange(half) * 3 // max(1, half), c["axes"] - 1).astype(np.int32)
    freq = THETA ** (-2.0 * np.arange(half) / c["rot"])
    return dict(op="rope", q=q, k=k, v=v, out=torch.empty((T, H, D), dtype=_type(c), device=_dev()),
                kc=_pool(c, g, n), vc=_pool(c, g, n), slots=_i32(slots), pos=_i32(_positions(c, r)),
                freq=torch.as_tensor(freq.astype(np.float32)).to(_dev()),
                axis=torch.as_tensor(axis), axis_dev=torch.as_tensor(axis.astype(np.int64)).to(_dev()),
                interleaved=c["interleaved"], fp8=c["kv"] == "fp8",
                err=torch.zeros(1, dtype=torch.int32, device=_dev()))


def _prepare_attention(c, seed):
    r = np.random.default_rng(seed)
    g = torch.Generator(device=_dev()).manual_seed(int(seed))
    if c["op"] == "decode":
        ctx = _decode_lens(c)
        q = np.ones_like(ctx)
    else:
        ctx, q = _chunk_lens(c)
    blocks = -(-ctx // c["block"])
    t, spare = _tables(r, blocks, int(blocks.max()), int(blocks.sum()) // 4 + 1)
    n = int(blocks.sum()) + len(spare)
    T, H, K, D = int(q.sum()), c["heads"], c["kv_heads"], c["dim"]
    kc, vc = _pool(c, g, n), _pool(c, g, n)
    s = dict(op=c["op"], query=torch.randn((T, H, D), generator=g, device=_dev(), dtype=_type(c)),
             out=torch.empty((T, H, D), dtype=_type(c), device=_dev()), kc=kc, vc=vc,
             tables=_i32(t), ctx=_i32(ctx), max_ctx=int(ctx.max()), max_rows=int(q.max()),
             start=_i32(np.concatenate([[0], np.cumsum(q)])), window=c["window"],
             sinks=c["sinks"], scale=D ** -0.5, fp8=c["kv"] == "fp8",
             kv_scale=FP8_SCALE if c["kv"] == "fp8" else 1.0,
             err=torch.zeros(1, dtype=torch.int32, device=_dev()))
    if c["op"] == "decode":
        s["partition"], s["workspace"] = c["partition"], None
        most = min(s["max_ctx"], -(-c["sinks"] // 16) * 16 + -(-c["window"] // 16) * 16 + 16)
        parts = -(-most // c["partition"]) if c["partition"] else 1
        if parts > 1:  # arrival counters, (m, l, o) of every partition, lengths
            size = (1 << 20) + 4 * c["seqs"] * (H * parts * (D + 2) + 1) + 2048
            s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=_dev())
    return s


def prepare(case, seed):
    if case["op"] == "maps":
        return _prepare_maps(case, seed)
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    return _prepare_attention(case, seed)


# ---------------------------------------------------------------------------
# the framework's calls

def _run_own(s):
    from paged_kv_cache_96_gb300 import binding as B
    if s["op"] == "maps":
        B.pa_build_step_maps(s["tables"], s["ctx"], s["new"], s["free"], s["count"], s["block"],
                             s["num_blocks"], s["start"], s["seq"], s["pos"], s["slot"],
                             s["ctx_out"], s["count_out"], error_word=s["err"])
        return {k: s[k] for k in ("tables", "free", "start", "seq", "pos", "slot", "ctx_out",
                                  "count_out")}
    if s["op"] == "rope":
        scale = FP8_SCALE if s["fp8"] else 1.0
        B.pa_rope_and_cache(s["out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"],
                            s["pos"], s["freq"], axis_of_pair=s["axis"],
                            interleaved=s["interleaved"], k_scale=scale, v_scale=scale,
                            error_word=s["err"])
        return _rope_outputs(s, s["out"])
    if s["op"] == "decode":
        B.pa_decode_attention_window(s["out"], s["query"], s["kc"], s["vc"], s["tables"],
                                     s["ctx"], s["max_ctx"], s["scale"], s["window"], s["sinks"],
                                     partition_size=s["partition"], workspace=s["workspace"],
                                     k_scale=s["kv_scale"], v_scale=s["kv_scale"],
                                     error_word=s["err"])
        return s["out"]
    B.pa_prefill_attention_window(s["out"], s["query"], s["kc"], s["vc"], s["tables"], s["start"],
                                  s["ctx"], s["max_ctx"], s["scale"], s["window"], s["sinks"],
                                  k_scale=s["kv_scale"], v_scale=s["kv_scale"],
                                  error_word=s["err"])
    return s["out"]


# ---------------------------------------------------------------------------
# the plain forms

def _rope_outputs(s, out):
    kc, vc = s["kc"], s["vc"]
    if s["fp8"]:
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    return {"query": out, "key_cache": kc, "value_cache": vc}


def _plain_maps(s):
    b, n = s["block"], s["num_blocks"]
    t, S, T = s["tables"], s["ctx"].shape[0], s["seq"].shape[0]
    ctx, q = s["ctx"].long(), s["new"].long()
    count = s["count"].long()
    gone = q < 0
    new = q.clamp(min=0)
    end = torch.where(gone, 0, ctx + new)
    have, want = (ctx + b - 1) // b, (end + b - 1) // b
    lb = torch.arange(t.shape[1], device=t.device)[None, :]
    # finished requests give their blocks back, in order, on top of the stack
    back = gone[:, None] & (lb < have[:, None])
    rank = torch.cumsum(back.reshape(-1), 0).reshape(back.shape) - 1
    given = back.sum()
    stack = torch.cat([s["free"].long(), torch.zeros(1, dtype=torch.int64, device=t.device)])
    at = torch.where(back, count + rank, n)
    stack = stack.scatter(0, at.reshape(-1), t.long().reshape(-1))[:n]
    # new blocks come off the top, requests in order
    need = torch.where(gone, 0, want - have)
    first = torch.cumsum(need, 0) - need
    take = (~gone)[:, None] & (lb >= have[:, None]) & (lb < want[:, None])
    top = count + given
    k = top - 1 - (first[:, None] + lb - have[:, None])
    tables = torch.where(take, stack[k.clamp(0, n - 1)], t.long())
    left = top - need.sum()
    idx = torch.arange(n, device=t.device)
    free = torch.where((idx >= count) & (idx < top), stack, s["free"].long())
    ends = torch.cumsum(new, 0)
    tok = torch.arange(T, device=t.device)
    seq = torch.searchsorted(ends, tok, right=True)
    real = tok < ends[-1]
    row = seq.clamp(max=S - 1)
    pos = ctx[row] + tok - (ends[row] - new[row])
    block = tables[row, (pos // b).clamp(0, t.shape[1] - 1)]
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"tables": i32(tables), "free": i32(free),
            "start": i32(torch.cat([torch.zeros_like(ends[:1]), ends])),
            "seq": i32(torch.where(real, seq, -1)), "pos": i32(torch.where(real, pos, -1)),
            "slot": i32(torch.where(real, block * b + pos % b, -1)), "ctx_out": i32(end),
            "count_out": i32(left)}


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, heads, D] in 32 bits; cos and sin [T, 1, rot / 2]."""
    y = x.clone()
    h = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, v
    else:
        y[..., :h], y[..., h:rot] = u, v
    return y


def _plain_rope(s):
    rot = 2 * s["freq"].shape[0]
    # angles of far positions need 64 bits
    angle = s["pos"][s["axis_dev"]].T.double() * s["freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(s["q"].float(), cos, sin, rot, s["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, rot, s["interleaved"])
    v = s["v"]
    kc, vc = (x.view(-1, *x.shape[2:]) for x in (s["kc"], s["vc"]))
    if s["fp8"]:
        inv = float(np.float32(1) / np.float32(FP8_SCALE))
        k, v = ((x.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x in (k, v))
    else:
        k = k.to(kc.dtype)
    # padding rows repeat the first row's write (the first row is never padding)
    at = s["slots"].long()
    pad = at < 0
    at = torch.where(pad, 0, at)
    keep = pad[:, None, None]
    at = torch.where(pad, at[0], at)
    kc[at] = torch.where(keep, k[:1], k)
    vc[at] = torch.where(keep, v[:1], v)
    return _rope_outputs(s, q)


def _values(pool, fp8, scale):
    return pool.view(torch.float8_e4m3fn).float() * scale if fp8 else pool.float()


def _gather(s, pool, pos):
    """Rows of one pool at positions pos [S, L] of each sequence, in 32 bits."""
    b = pool.shape[1]
    p = pos.clamp(min=0)
    block = torch.gather(s["tables"].long(), 1, (p // b).clamp(max=s["tables"].shape[1] - 1))
    return _values(pool.view(-1, *pool.shape[2:])[block * b + p % b], s["fp8"], s["kv_scale"])


def _plain_decode(s):
    ctx = s["ctx"].long()[:, None]
    i = torch.arange(s["sinks"] + min(s["window"], s["max_ctx"]), device=ctx.device)[None, :]
    low = (ctx - s["window"]).clamp(min=0)  # first position of the window
    sink = i < s["sinks"]
    pos = torch.where(sink, i, low + i - s["sinks"])
    seen = torch.where(sink, pos < torch.minimum(low, ctx), pos < ctx)
    k, v = _gather(s, s["kc"], pos), _gather(s, s["vc"], pos)
    S, L, K, D = k.shape
    q = s["query"].float().view(S, K, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / e.sum(-1, keepdim=True)
    return o.reshape(s["query"].shape).to(s["query"].dtype)


def _plain_chunk(s):
    start, ctx = s["start"].long(), s["ctx"].long()
    rows = start[1:] - start[:-1]
    first = ctx - rows  # position of each chunk's first row
    R, W, N = s["max_rows"], s["window"], s["sinks"]
    dev = ctx.device
    # the chunk's keys: the first tokens, then the window of the first row on
    low = (first + 1 - W).clamp(min=0)[:, None]
    i = torch.arange(N + min(W + R, s["max_ctx"]), device=dev)[None, :]
    pos = torch.where(i < N, i, low + i - N)
    live = torch.where(i < N, pos < torch.minimum(low, ctx[:, None]), pos < ctx[:, None])
    k, v = _gather(s, s["kc"], pos), _gather(s, s["vc"], pos)
    S, L, K, D = k.shape
    j = torch.arange(R, device=dev)[None, :]
    row = (start[:-1, None] + j).clamp(max=s["query"].shape[0] - 1)
    at = first[:, None] + j  # [S, R] position of each row
    q = s["query"][row].float().view(S, R, K, -1, D).permute(0, 2, 3, 1, 4).reshape(S, K, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    p, a = pos[:, None, :], at[:, :, None]
    seen = live[:, None, :] & (p <= a) & ((p < N) | (p > a - W))
    x = x.view(S, K, -1, R, L).masked_fill_(~seen[:, None, None], -math.inf)
    e = x.sub_(x.amax(-1, keepdim=True)).exp_()
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(S, K, -1, L), v.permute(0, 2, 1, 3)).view(S, K, -1, R, D) / z
    o = o.permute(0, 3, 1, 2, 4).reshape(S, R, -1, D)
    return o[j < rows[:, None]].to(s["query"].dtype)


def run(state):
    if own:
        return _run_own(state)
    return {"maps": _plain_maps, "rope": _plain_rope, "decode": _plain_decode,
            "chunk": _plain_chunk}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, row by row

def _exact_rope(c, s):
    rot, T = c["rot"], c["tokens"]
    angle = np.zeros((T, rot // 2))
    freq, pos, axis = s["freq"].cpu().numpy(), s["pos"].cpu().numpy(), s["axis"].numpy()
    for i in range(rot // 2):
        angle[:, i] = pos[axis[i]].astype(np.float64) * float(freq[i])
    w = torch.polar(torch.ones(T, rot // 2, dtype=torch.float64), torch.as_tensor(angle)).to(_dev())

    def turn(x):  # each pair as a complex number
        x = x.double()
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], -1, 2).contiguous())
            r = torch.view_as_real(z * w[:, None]).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * w[:, None]
            r = torch.cat([z.real, z.imag], -1)
        return torch.cat([r, x[..., rot:]], -1)

    def cached(pool, x):
        if s["fp8"]:
            flat = pool.view(torch.float8_e4m3fn).double().flatten(0, 1)
            x = (x.double() / FP8_SCALE).clamp(-448, 448)
        else:
            flat = pool.double().flatten(0, 1)
        real = s["slots"] >= 0
        flat[s["slots"][real].long()] = x[real].double()
        return flat.view(pool.shape)

    return {"query": turn(s["q"]), "key_cache": cached(s["kc"], turn(s["k"])),
            "value_cache": cached(s["vc"], s["v"])}


def _exact_attention(c, s):
    start, ctx, tables = s["start"].tolist(), s["ctx"].tolist(), s["tables"].cpu().numpy()
    H, K, D, b = c["heads"], c["kv_heads"], c["dim"], c["block"]
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device=_dev())
    for i, n in enumerate(ctx):
        lo, hi = start[i], start[i + 1]
        p = np.arange(n)
        slot = torch.as_tensor(tables[i][p // b].astype(np.int64) * b + p % b).to(_dev())
        at = torch.arange(n - (hi - lo), n, device=_dev())[:, None]
        key = torch.arange(n, device=_dev())[None, :]
        hide = (key > at) | ((key <= at - c["window"]) & (key >= c["sinks"]))
        for h in range(K):
            k, v = ((x.view(torch.float8_e4m3fn) if s["fp8"] else x)[:, :, h].flatten(0, 1)[slot]
                    .double() * s["kv_scale"] for x in (s["kc"], s["vc"]))
            for r in range(lo, hi, 512):  # a slab of rows at a time
                e = min(hi, r + 512)
                heads = slice(h * (H // K), (h + 1) * (H // K))
                q = s["query"][r:e, heads].double()
                x = torch.einsum("rgd,nd->rgn", q, k) * s["scale"]
                x = x.masked_fill(hide[r - lo:e - lo, None, :], -math.inf)
                out[r:e, heads] = torch.einsum("rgn,nd->rgd", torch.softmax(x, -1), v)
    return out


def exact(case, seed):
    if case["op"] == "maps":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    ctx, q = (_decode_lens(case), 1) if case["op"] == "decode" else _chunk_lens(case)
    if 4 * float((ctx * q).sum()) * case["heads"] * case["dim"] > 1e13:
        return None
    return _exact_attention(case, s)
