"""Measured cases of the operators that let a long context be read in part or kept in part.

Five operators over the paged KV cache:

  summary  8-bit bounds of the keys of every block that a step wrote to
           (``pa_summarize_blocks``)
  select   the blocks that each query row attends, by the largest score that
           their bounds allow (``pa_select_blocks``)
  sparse   attention of each row over its selected blocks
           (``pa_decode_attention_sparse``)
  weights  decode attention that also adds what each cached token was attended
           with to its accumulated weight (``pa_decode_attention_weights``)
  evict    sequences over a limit cut down to the tokens of largest accumulated
           weight: the plan, and the cache rows moved by it
           (``pa_plan_eviction``, ``pa_move_tokens``)

Lengths are drawn from a case's own ``lens`` number, so that its work is known
from the case alone; values, block placement and selections come from the seed
of ``prepare``.  Pools hold finite values everywhere, as a pool whose blocks
were used before does.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

FP8_SCALE = 0.0137  # per-pool scale of e4m3 codes, N(0, 1) values
LEVELS = 127.0      # codes of a block's bounds
TINY = 2.0 ** -40   # amplitudes below it count as zero


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # four short chats on a small model, one new token each
        dict(name="summary decode 4 d64", op="summary", seqs=4, kv_heads=4, dim=64, block=16,
             dtype="f16", kv="same", min_ctx=1, max_ctx=500, new=1, lens=51),
        # whole contexts, as after a prompt or an eviction: a GQA 70B-like layer
        dict(name="summary rebuild 128", op="summary", seqs=128, kv_heads=8, dim=128, block=16,
             dtype="bf16", kv="same", min_ctx=16, max_ctx=8192, new=0, lens=52),
        # a decode step of a GQA 70B-like layer: 64 blocks of 16 tokens a head
        dict(name="select decode gqa", op="select", seqs=128, rows=1, pad=0, heads=64, kv_heads=8,
             dim=128, block=16, dtype="bf16", top_k=64, first=1, last=2, min_ctx=16, max_ctx=8192,
             lens=53),
        # few requests with very long contexts, drafted tokens behind each
        dict(name="select long 131072", op="select", seqs=8, rows=3, pad=2, heads=32, kv_heads=8,
             dim=128, block=32, dtype="f16", top_k=128, first=1, last=4, min_ctx=2000,
             max_ctx=131072, lens=54),
        # four short chats on a small model
        dict(name="sparse 4 rows d64", op="sparse", seqs=4, rows=1, pad=0, heads=4, kv_heads=4,
             dim=64, block=16, dtype="f16", kv="same", top_k=8, min_ctx=1, max_ctx=500,
             partition=0, lens=55),
        # the decode step of the third case
        dict(name="sparse decode gqa", op="sparse", seqs=128, rows=1, pad=0, heads=64, kv_heads=8,
             dim=128, block=16, dtype="bf16", kv="same", top_k=64, min_ctx=16, max_ctx=8192,
             partition=1024, lens=53),
        # long contexts over an FP8 cache, few requests, the list split
        dict(name="sparse long fp8", op="sparse", seqs=16, rows=1, pad=0, heads=32, kv_heads=8,
             dim=128, block=32, dtype="bf16", kv="fp8", top_k=128, min_ctx=64, max_ctx=32768,
             partition=512, lens=56),
        # four short chats on a small model
        dict(name="weights 4 d64", op="weights", seqs=4, heads=4, kv_heads=4, dim=64, block=16,
             dtype="f16", kv="same", min_ctx=1, max_ctx=500, partition=0, lens=57),
        # a GQA 70B-like decode layer, 128 requests
        dict(name="weights decode gqa", op="weights", seqs=128, heads=64, kv_heads=8, dim=128,
             block=16, dtype="bf16", kv="same", min_ctx=16, max_ctx=8192, partition=1024,
             lens=58),
        # long contexts over an FP8 cache, few requests
        dict(name="weights long fp8", op="weights", seqs=16, heads=32, kv_heads=8, dim=128,
             block=32, dtype="bf16", kv="fp8", min_ctx=64, max_ctx=32768, partition=512, lens=59),
        # a small model's chats, two of them over their limit
        dict(name="evict 5 d64", op="evict", seqs=5, kv_heads=4, dim=64, block=16, dtype="f16",
             kv="same", limit=256, budget=192, sinks=4, recent=32, min_ctx=1, max_ctx=500,
             lens=60),
        # a server that halves what passes 4096 tokens, GQA 70B-like layer
        dict(name="evict 128", op="evict", seqs=128, kv_heads=8, dim=128, block=16, dtype="bf16",
             kv="same", limit=4096, budget=2048, sinks=4, recent=512, min_ctx=64, max_ctx=8192,
             lens=61),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["summary", "select", "sparse", "weights", "evict"])
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 16])
    c = dict(op=op, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32, 64]),
             dtype=rng.choice(["f16", "bf16"]), min_ctx=1, lens=rng.randrange(1, 1 << 30))
    wide = kv_heads * dim / 1024  # of the largest cases' rows
    if op == "select":
        c.update(seqs=_log(rng, 1, 128), rows=rng.choice([1, 1, 2, 3]), pad=rng.choice([0, 2]))
        room = int(24 * 131072 / (c["seqs"] * c["rows"] * wide * max(1, heads / kv_heads / 4)))
        c.update(heads=heads, max_ctx=_log(rng, 32 * c["block"], min(131072, room)))
        c["top_k"] = _log(rng, 4, min(128, c["max_ctx"] // (4 * c["block"])))
        c.update(first=rng.randint(0, min(2, c["top_k"] - 2)), last=rng.randint(1, 2))
        return c
    c["kv"] = rng.choice(["same", "same", "fp8"])
    if op == "summary":
        c.update(seqs=_log(rng, 1, 256), new=rng.choice([0, 1, _log(rng, 2, 600)]))
        c["max_ctx"] = _log(rng, 100, min(8192, int(2 * 131072 / (c["seqs"] * wide))))
        return c
    if op == "sparse":
        c.update(seqs=_log(rng, 1, 128), rows=rng.choice([1, 1, 2]), pad=rng.choice([0, 3]))
        room = int(128 * 1024 / (c["seqs"] * c["rows"] * wide * c["block"]))
        c.update(heads=heads, top_k=_log(rng, 2, max(3, min(128, room))),
                 max_ctx=_log(rng, 64, 32768), partition=rng.choice([0, 256, 512, 1024]))
        return c
    c["seqs"] = _log(rng, 1, 128)
    room = int(128 * 2048 / (c["seqs"] * wide))
    if op == "weights":
        c.update(heads=heads, max_ctx=_log(rng, 64, min(32768, room)),
                 partition=rng.choice([0, 256, 512, 1024]))
        if c["partition"] == 0 and c["seqs"] * kv_heads < 64:
            c["partition"] = 256
        return c
    c["max_ctx"] = _log(rng, 100, min(16384, room))
    c["budget"] = max(24, int(c["max_ctx"] * rng.uniform(0.1, 0.8)))
    c["limit"] = c["budget"] + rng.choice([0, rng.randint(0, c["max_ctx"] // 8)])
    c.update(sinks=rng.choice([0, rng.randint(1, 8)]), recent=rng.randint(1, c["budget"] // 2))
    return c


# ---------------------------------------------------------------------------
# lengths (from the case alone) and work

def _lens(c):
    r = np.random.default_rng(c["lens"])
    hi, lo = c["max_ctx"], min(c["min_ctx"], c["max_ctx"])
    x = np.exp(r.normal(math.log(max(lo, hi / 3)), 0.8, size=c["seqs"]))
    x = np.clip(np.rint(x), lo, hi).astype(np.int64)
    x[0] = hi
    return np.maximum(x, c.get("rows", 1))


def _new(c, ctx):
    """New tokens of each sequence (a whole context where new is 0)."""
    return np.minimum(ctx, c["new"]) if c["new"] else ctx


def _moved(c, ctx):
    """Tokens that an eviction moves, on average over weights of one distribution."""
    over = ctx[ctx > c["limit"]].astype(np.float64)
    guarded = c["sinks"] + c["recent"]
    share = (c["budget"] - guarded) / np.maximum(1, over - guarded)
    recent = np.minimum(c["recent"], over - c["budget"])
    return int(np.sum(recent + share * np.maximum(0, over - c["recent"] - c["budget"])))


def work(case):
    c = case
    ctx = _lens(c)
    K, D, b = c["kv_heads"], c["dim"], c["block"]
    e = 1 if c.get("kv") == "fp8" else 2
    if c["op"] == "summary":
        first = (ctx - _new(c, ctx)) // b
        blocks = int((-(-ctx // b) - first).sum())
        tokens = int((ctx - first * b).sum())
        return {"bytes": tokens * K * D * e + blocks * (K * (2 * D + 4) + 4),
                "flops": 2 * tokens * K * D}
    if c["op"] == "evict":
        over = ctx[ctx > c["limit"]]
        row = 2 * K * D * e + 4
        return {"bytes": int(4 * ctx.sum() + 4 * np.minimum(ctx, c["budget"]).sum() +
                             2 * _moved(c, ctx) * row + 8 * len(over) * c["budget"]),
                "flops": 0}
    H = c["heads"]
    if c["op"] == "weights":
        n = int(ctx.sum())
        return {"bytes": n * (2 * K * D * e + 8) + 4 * c["seqs"] * H * D, "flops": 4 * n * H * D}
    T = c["seqs"] * c["rows"] + c["pad"]
    blocks = -(-ctx // b)
    if c["op"] == "select":
        n = int(blocks.sum())
        return {"bytes": n * (K * (2 * D + 4) + 4) + 2 * T * H * D + 4 * T * K * c["top_k"],
                "flops": 4 * n * c["rows"] * H * D}
    read = int(np.minimum(blocks, c["rows"] * c["top_k"]).sum()) * b
    seen = int(np.minimum(blocks, c["top_k"]).sum()) * b * c["rows"]
    return {"bytes": 2 * read * K * D * e + 4 * T * H * D + 4 * T * K * c["top_k"],
            "flops": 4 * seen * H * D}


# ---------------------------------------------------------------------------
# inputs

def _dev():
    return torch.device("cuda")


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).to(_dev())


def _type(c):
    return torch.float16 if c["dtype"] == "f16" else torch.bfloat16


def _tables(r, blocks):
    """A shuffled placement: block_tables [S, most] (unused entries 0), pool size."""
    total, width = int(blocks.sum()), int(blocks.max())
    spare = total // 4 + 1
    ids = r.permutation(total + spare).astype(np.int32)
    t = np.zeros((len(blocks), width), dtype=np.int32)
    t[np.arange(width)[None, :] < blocks[:, None]] = ids[:total]
    return t, total + spare, ids[total:]


def _pool(c, g, num_blocks):
    shape = (num_blocks, c["block"], c["kv_heads"], c["dim"])
    x = torch.randn(shape, generator=g, device=_dev(),
                    dtype=torch.float32 if c["kv"] == "fp8" else _type(c))
    if c["kv"] == "fp8":
        return (x / FP8_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def _rows(c, ctx):
    """Sequence and position of each query row: the last `rows` tokens of every
    sequence, then padding rows."""
    seq = np.repeat(np.arange(c["seqs"]), c["rows"])
    pos = np.repeat(ctx - c["rows"], c["rows"]) + np.tile(np.arange(c["rows"]), c["seqs"])
    pad = np.full(c["pad"], -1)
    return np.concatenate([seq, pad]), np.concatenate([pos, pad])


def prepare(case, seed):
    c = case
    r = np.random.default_rng(seed)
    g = torch.Generator(device=_dev()).manual_seed(int(seed))
    ctx = _lens(c)
    blocks = -(-ctx // c["block"])
    t, n, spare = _tables(r, blocks)
    K, D, S, b = c["kv_heads"], c["dim"], c["seqs"], c["block"]
    fp8 = c.get("kv") == "fp8"
    s = dict(op=c["op"], tables=_i32(t), ctx=_i32(ctx), max_ctx=int(ctx.max()), block=b,
             fp8=fp8, kv_scale=FP8_SCALE if fp8 else 1.0,
             err=torch.zeros(1, dtype=torch.int32, device=_dev()))
    if c["op"] == "summary":
        start = np.concatenate([[0], np.cumsum(_new(c, ctx))])
        most = int((blocks - (ctx - _new(c, ctx)) // b).max())
        s.update(kc=_pool(c, g, n), start=_i32(start), whole=c["new"] == 0, most=most,
                 codes=torch.zeros((n, K, 2, D), dtype=torch.int8, device=_dev()),
                 scales=torch.zeros((n, K), device=_dev()))
        return s
    if c["op"] == "evict":
        # a heavy tail, as accumulated attention has, and tokens that nothing attended
        w = torch.exp(1.5 * torch.randn((n, b), generator=g, device=_dev()))
        w[torch.rand((n, b), generator=g, device=_dev()) < 0.02] = 0.0
        free = np.full(n, -1, dtype=np.int32)
        free[:len(spare)] = spare
        moves = max(1, min(c["budget"], s["max_ctx"] - c["budget"]))
        s.update(kc=_pool(c, g, n), vc=_pool(c, g, n), weights=w, weights_out=torch.zeros_like(w),
                 free=_i32(free), count=_i32([len(spare)]), count_out=_i32([0]),
                 ctx_out=_i32(np.zeros(S)), limit=c["limit"], budget=c["budget"],
                 sinks=c["sinks"], recent=c["recent"],
                 moves=torch.full((S, moves, 2), -1, dtype=torch.int32, device=_dev()))
        return s
    H = c["heads"]
    if c["op"] == "weights":
        from_ = ctx - 1  # tokens with a weight so far: all but the new one
        from_[1::5] = 0  # none, for a context that no step has attended
        w = torch.exp(1.5 * torch.randn((n, b), generator=g, device=_dev()))
        T = S
        parts = -(-s["max_ctx"] // c["partition"]) if c["partition"] else 1
        size = (1 << 20) + 4 * S * H * parts * (D + 2) + 4 * S * H * (s["max_ctx"] + 16) + \
            8 * S * H + 65536
        s.update(kc=_pool(c, g, n), vc=_pool(c, g, n), weights=w, weights_out=torch.zeros_like(w),
                 weighted=_i32(from_), partition=c["partition"], scale=D ** -0.5,
                 workspace=torch.zeros(size, dtype=torch.uint8, device=_dev()))
    else:
        seq, pos = _rows(c, ctx)
        T = len(seq)
        s.update(seq=_i32(seq), pos=_i32(pos))
    s["query"] = torch.randn((T, H, D), generator=g, device=_dev(), dtype=_type(c))
    if c["op"] == "select":
        # bounds of 16 or more N(0, 1) keys around a block's own mean
        mean = 0.4 * torch.randn((n, K, 1, D), generator=g, device=_dev())
        side = torch.tensor([-1.7, 1.7], device=_dev())[:, None]
        x = mean + side + 0.4 * torch.randn((n, K, 2, D), generator=g, device=_dev())
        top = x.abs().amax((2, 3))
        s.update(codes=torch.round(x / top[..., None, None] * LEVELS).to(torch.int8),
                 scales=top / LEVELS, first=c["first"], last=c["last"],
                 selected=torch.zeros((T, K, c["top_k"]), dtype=torch.int32, device=_dev()))
        return s
    s["out"] = torch.empty_like(s["query"])
    if c["op"] == "weights":
        return s
    # sparse: the newest block and others at random, in ascending order
    have = _i32(np.where(seq < 0, 0, pos // b + 1)).long()[:, None, None]
    u = torch.rand((T, K, int(blocks.max())), generator=g, device=_dev())
    i = torch.arange(u.shape[2], device=_dev())
    u = u.masked_fill(i == have - 1, 2.0).masked_fill(i >= have, -1.0)
    k = min(c["top_k"], u.shape[2])
    best = u.topk(k, -1)
    pick = best.indices.masked_fill(best.values < 0, 1 << 30).sort(-1).values
    chosen = torch.full((T, K, c["top_k"]), -1, dtype=torch.int32, device=_dev())
    chosen[:, :, :k] = pick.masked_fill(pick == 1 << 30, -1).to(torch.int32)
    s.update(kc=_pool(c, g, n), vc=_pool(c, g, n), chosen=chosen, partition=c["partition"],
             scale=D ** -0.5, workspace=None)
    parts = -(-c["top_k"] * b // c["partition"]) if c["partition"] else 1
    if parts > 1:  # arrival counters, (m, l, o) of every partition, lengths
        size = (1 << 20) + 4 * T * (H * parts * (D + 2) + K + 1) + 4096
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=_dev())
    return s


# ---------------------------------------------------------------------------
# the framework's calls

def _pools(s):
    kc, vc = s["kc"], s["vc"]
    if s["fp8"]:
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    return {"key_cache": kc, "value_cache": vc}


def _plan_outputs(s):
    return {k: s[k] for k in ("moves", "ctx_out", "free", "count_out", "weights_out")}


def _run_own(s):
    from paged_kv_cache_96_gb300 import binding as B
    if s["op"] == "summary":
        B.pa_summarize_blocks(s["codes"], s["scales"], s["kc"], s["tables"], s["ctx"],
                              query_start=None if s["whole"] else s["start"],
                              error_word=s["err"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if s["op"] == "select":
        B.pa_select_blocks(s["selected"], s["query"], s["codes"], s["scales"], s["tables"],
                           s["seq"], s["pos"], s["max_ctx"], s["block"], num_first=s["first"],
                           num_last=s["last"], error_word=s["err"])
        return s["selected"]
    if s["op"] == "sparse":
        B.pa_decode_attention_sparse(s["out"], s["query"], s["kc"], s["vc"], s["tables"],
                                     s["seq"], s["pos"], s["chosen"], s["scale"],
                                     partition_size=s["partition"], workspace=s["workspace"],
                                     k_scale=s["kv_scale"], v_scale=s["kv_scale"],
                                     error_word=s["err"])
        return s["out"]
    if s["op"] == "weights":
        B.pa_decode_attention_weights(s["out"], s["weights_out"], s["query"], s["kc"], s["vc"],
                                      s["weights"], s["tables"], s["ctx"], s["weighted"],
                                      s["max_ctx"], s["scale"], s["workspace"],
                                      partition_size=s["partition"], k_scale=s["kv_scale"],
                                      v_scale=s["kv_scale"], error_word=s["err"])
        return {"out": s["out"], "weights": s["weights_out"]}
    B.pa_plan_eviction(s["moves"], s["ctx_out"], s["count_out"], s["weights_out"], s["tables"],
                       s["ctx"], s["weights"], s["free"], s["count"], s["max_ctx"], s["limit"],
                       s["budget"], s["sinks"], s["recent"], error_word=s["err"])
    B.pa_move_tokens(s["kc"], s["vc"], s["moves"], error_word=s["err"])
    return {**_plan_outputs(s), **_pools(s)}


# ---------------------------------------------------------------------------
# the plain forms

def _values(pool, fp8, scale=1.0):
    return pool.view(torch.float8_e4m3fn).float() * scale if fp8 else pool.float()


def _slots(s, pos):
    """Slots of positions [S, ...] of each sequence (clamped into its table)."""
    b, t = s["block"], s["tables"].long()
    p = pos.clamp(min=0)
    i = (p // b).clamp(max=t.shape[1] - 1)
    return torch.gather(t, 1, i.flatten(1)).view(i.shape) * b + p % b


def _plain_summary(s):
    kc, b = s["kc"], s["block"]
    ctx = s["ctx"].long()[:, None]
    new = ctx if s["whole"] else (s["start"][1:] - s["start"][:-1]).long()[:, None]
    last = (ctx - 1) // b
    i = last - torch.arange(s["most"], device=kc.device)
    touched = (i >= 0) & (i >= (ctx - new) // b)
    # blocks outside the step repeat the first sequence's last one
    row = torch.where(touched, torch.arange(len(ctx), device=kc.device)[:, None], 0)
    blk = torch.where(touched, i, last[0])
    phys = s["tables"].long()[row, blk]
    live = blk[..., None] * b + torch.arange(b, device=kc.device) < ctx[row, 0][..., None]
    x = _values(kc[phys], s["fp8"])
    gone = ~live[..., None, None]
    lo = x.masked_fill(gone, math.inf).amin(2)
    hi = x.masked_fill(gone, -math.inf).amax(2)
    bounds = torch.stack([lo, hi], -2)
    top = bounds.abs().amax((-1, -2))
    good = torch.isfinite(top)
    some = good & (top >= TINY)
    inv = torch.where(some, torch.full_like(top, LEVELS) / torch.where(some, top, 1.0), 0.0)
    codes = torch.round(torch.where(good[..., None, None], bounds, 0.0) * inv[..., None, None])
    scale = torch.where(some, top * torch.full_like(top, 1.0 / LEVELS), 0.0)
    s["codes"][phys] = codes.clamp(-LEVELS, LEVELS).to(torch.int8)
    s["scales"][phys] = torch.where(good, scale, math.inf)
    return {"codes": s["codes"], "scales": s["scales"]}


def _plain_select(s):
    T, K, top_k = s["selected"].shape
    b = s["block"]
    pos = torch.where(s["seq"] < 0, -1, s["pos"]).long()
    have = torch.div(pos + b, b, rounding_mode="floor")[:, None]  # blocks of each row
    n = s["tables"].shape[1]
    i = torch.arange(n, device=pos.device)
    phys = s["tables"].long()[s["seq"].long().clamp(min=0)]
    q = s["query"].float().view(T, K, -1, s["query"].shape[2])
    top = q.abs().amax(-1, keepdim=True)
    some = torch.isfinite(top) & (top >= TINY)
    inv = torch.where(some, torch.full_like(top, LEVELS) / torch.where(some, top, 1.0), 0.0)
    q = torch.round(torch.where(some, q, 0.0) * inv).clamp(-LEVELS, LEVELS)
    q_scale = torch.where(some, top * torch.full_like(top, 1.0 / LEVELS), 0.0)
    # whole numbers below 2^24: exact in 32 bits, in any order
    bounds = s["codes"][phys].float().permute(0, 2, 3, 4, 1)  # [T, K, 2, D, n]
    x = torch.matmul(q.clamp(max=0), bounds[:, :, 0]) + torch.matmul(q.clamp(min=0),
                                                                     bounds[:, :, 1])
    scale = s["scales"][phys].transpose(1, 2)
    best = (x * q_scale).amax(2)
    score = torch.where(torch.isinf(scale), scale, best * torch.where(torch.isinf(scale), 0.0,
                                                                      scale))
    bits = score.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    h = have[..., None]
    key = key.masked_fill((i < s["first"]) | (i >= h - s["last"]), 1 << 40)
    key = key.masked_fill(i >= h, -(1 << 40))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :top_k]
    order = torch.where(order < h, order, n + 1).sort(-1).values
    out = torch.full_like(s["selected"], -1)
    out[..., :order.shape[-1]] = torch.where(order > n, -1, order).to(torch.int32)
    return out


def _plain_sparse(s):
    T, K, top_k = s["chosen"].shape
    kc, vc, b = s["kc"], s["vc"], s["block"]
    D, dev = kc.shape[3], kc.device
    blk = s["chosen"].long()
    p = blk[..., None] * b + torch.arange(b, device=dev)
    seen = (blk[..., None] >= 0) & (p <= s["pos"].long()[:, None, None, None])
    seen = (seen & (s["seq"] >= 0)[:, None, None, None]).view(T, K, 1, -1)
    phys = s["tables"].long()[s["seq"].long().clamp(min=0)[:, None, None], blk.clamp(min=0)]
    slot = (phys[..., None] * b + torch.arange(b, device=dev)).view(T, K, -1)
    head = torch.arange(K, device=dev)[:, None]
    k, v = (_values(x.view(-1, K, D)[slot, head], s["fp8"], s["kv_scale"]) for x in (kc, vc))
    q = s["query"].float().view(T, K, -1, D)
    x = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(z == 0, 1.0, z)
    return o.reshape(s["query"].shape).to(s["query"].dtype)


def _plain_weights(s):
    kc, vc = s["kc"], s["vc"]
    ctx = s["ctx"].long()[:, None]
    p = torch.arange(s["max_ctx"], device=kc.device)[None, :].expand(ctx.shape[0], -1)
    seen = p < ctx
    slot = _slots(s, p)
    K, D = kc.shape[2:]
    k, v = (_values(x.view(-1, K, D)[slot], s["fp8"], s["kv_scale"]) for x in (kc, vc))
    q = s["query"].float().view(len(ctx), K, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    x = x.masked_fill_(~seen[:, None, None, :], -math.inf)
    e = x.sub_(x.amax(-1, keepdim=True)).exp_()
    e /= e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)).reshape(s["query"].shape).to(s["query"].dtype)
    before = s["weights"].view(-1)[slot]
    after = torch.where(p < s["weighted"][:, None], before, 0.0) + e.sum((1, 2))
    # positions past the context repeat its first token
    at = torch.where(seen, slot, slot[:, :1])
    s["weights_out"].view(-1)[at] = torch.where(seen, after, after[:, :1])
    return {"out": o, "weights": s["weights_out"]}


def _plain_evict(s):
    ctx, b, dev = s["ctx"].long()[:, None], s["block"], s["ctx"].device
    budget, n = s["budget"], s["free"].shape[0]
    p = torch.arange(s["max_ctx"], device=dev)[None, :].expand(ctx.shape[0], -1)
    over = ctx > s["limit"]
    slot = _slots(s, p)
    w = s["weights"].view(-1)[slot]
    guarded = (p < s["sinks"]) | (p >= ctx - s["recent"])
    key = torch.where(w > 0, w, 0.0).masked_fill(guarded, math.inf).masked_fill(p >= ctx, -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :budget]
    kept = torch.zeros_like(guarded).scatter_(1, order, True) & over
    hole = over & ~kept & (p < budget)
    late = kept & (p >= budget)
    # the i-th kept token past the budget takes the place of the i-th evicted before it
    M = s["moves"].shape[1]
    at = lambda m: torch.where(m, torch.cumsum(m, 1) - 1, M).clamp(max=M)  # noqa: E731
    moves = torch.full((len(ctx), M + 1, 2), -1, dtype=torch.int64, device=dev)
    moves[..., 0].scatter_(1, at(late), slot.masked_fill(~late, -1))
    moves[..., 1].scatter_(1, at(hole), slot.masked_fill(~hole, -1))
    moves = moves[:, :M]
    src, dst = moves.reshape(-1, 2).unbind(1)
    real = dst >= 0
    # entries without a move repeat the first one (or leave slot 0 as it is)
    one = torch.argmax(real.to(torch.int8))
    any_ = real[one]
    src = torch.where(real, src, torch.where(any_, src[one], 0))
    dst = torch.where(real, dst, torch.where(any_, dst[one], 0))
    end = torch.where(over, budget, ctx)
    out = s["weights_out"].view(-1)
    stay = p < end
    out[torch.where(stay, slot, slot[:, :1])] = torch.where(stay, w, w[:, :1])
    out[torch.where(real, dst, torch.where(any_, dst[one], slot[0, 0]))] = \
        torch.where(any_, s["weights"].view(-1)[src], out[slot[0, 0]])
    kc, vc = s["kc"].view(n * b, -1), s["vc"].view(n * b, -1)
    kc[dst], vc[dst] = kc[src], vc[src]
    # blocks behind the budget go back on the stack, in order
    t = s["tables"].long()
    i = torch.arange(t.shape[1], device=dev)[None, :]
    back = over & (i >= (end + b - 1) // b) & (i < (ctx + b - 1) // b)
    count = s["count"].long()
    put = torch.where(back, count + torch.cumsum(back.view(-1), 0).view(back.shape) - 1, n)
    stack = torch.cat([s["free"].long(), torch.zeros(1, dtype=torch.int64, device=dev)])
    stack = stack.scatter(0, put.view(-1), t.view(-1))[:n]
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"moves": i32(moves), "ctx_out": i32(end[:, 0]), "free": i32(stack),
            "count_out": i32(count + back.sum()), "weights_out": s["weights_out"], **_pools(s)}


def run(state):
    if own:
        return _run_own(state)
    return {"summary": _plain_summary, "select": _plain_select, "sparse": _plain_sparse,
            "weights": _plain_weights, "evict": _plain_evict}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence

def _exact_summary(c, s):
    scales = s["scales"].double()
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    tables, b = s["tables"].cpu().numpy(), c["block"]
    pool = s["kc"].view(torch.float8_e4m3fn) if s["fp8"] else s["kc"]
    for i, n in enumerate(ctx):
        new = start[i + 1] - start[i]
        for j in range((n - new) // b, -(-n // b)):
            at = int(tables[i, j])
            x = pool[at, :min(b, n - j * b)].double()
            scales[at] = x.abs().amax((0, 2)) / LEVELS
    return {"codes": None, "scales": scales}


def _exact_rows(c, s):
    seq, pos = s["seq"].tolist(), s["pos"].tolist()
    tables, chosen = s["tables"].cpu().numpy(), s["chosen"].cpu().numpy()
    K, b = c["kv_heads"], c["block"]
    G = c["heads"] // K
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device=_dev())
    for t, (i, at) in enumerate(zip(seq, pos)):
        for h in range(K if i >= 0 else 0):
            blk = chosen[t, h][chosen[t, h] >= 0]
            p = (blk[:, None] * b + np.arange(b)).reshape(-1)
            p = p[p <= at]
            where = torch.as_tensor(tables[i][p // b].astype(np.int64) * b + p % b).to(_dev())
            k, v = ((x.view(torch.float8_e4m3fn) if s["fp8"] else x).flatten(0, 1)[where, h]
                    .double() * s["kv_scale"] for x in (s["kc"], s["vc"]))
            x = s["query"][t, h * G:(h + 1) * G].double() @ k.T * s["scale"]
            out[t, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return out


def _exact_weights(c, s):
    tables, b = s["tables"].cpu().numpy(), c["block"]
    K = c["kv_heads"]
    G = c["heads"] // K
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device=_dev())
    total = s["weights_out"].double().flatten()
    before = s["weights"].double().flatten()
    weighted = s["weighted"].tolist()
    for i, n in enumerate(s["ctx"].tolist()):
        p = np.arange(n)
        slot = torch.as_tensor(tables[i][p // b].astype(np.int64) * b + p % b).to(_dev())
        total[slot] = torch.where(torch.arange(n, device=_dev()) < weighted[i], before[slot], 0.0)
        for h in range(K):
            k, v = ((x.view(torch.float8_e4m3fn) if s["fp8"] else x).flatten(0, 1)[slot, h]
                    .double() * s["kv_scale"] for x in (s["kc"], s["vc"]))
            w = torch.softmax(s["query"][i, h * G:(h + 1) * G].double() @ k.T * s["scale"], -1)
            out[i, h * G:(h + 1) * G] = w @ v
            total[slot] += w.sum(0)
    return {"out": out, "weights": total.view(s["weights"].shape)}


def _exact_evict(c, s):
    """The weights of what stays; the rest is whole numbers and rows as they were."""
    tables, b = s["tables"].cpu().numpy(), c["block"]
    w = s["weights"].double().flatten().cpu().numpy()
    out = s["weights_out"].double().flatten().cpu().numpy()
    for i, n in enumerate(s["ctx"].tolist()):
        p = np.arange(n)
        slot = tables[i][p // b].astype(np.int64) * b + p % b
        if n <= c["limit"]:
            out[slot] = w[slot]
            continue
        middle = p[c["sinks"]:n - c["recent"]]
        rank = np.lexsort((middle, -w[slot[middle]]))
        gone = np.sort(middle[rank[c["budget"] - c["sinks"] - c["recent"]:]])
        kept = np.setdiff1d(p, gone)
        place = kept.copy()
        place[kept >= c["budget"]] = gone[gone < c["budget"]]
        out[slot[place]] = w[slot[kept]]
    return {"moves": None, "ctx_out": None, "free": None, "count_out": None,
            "weights_out": torch.as_tensor(out).view(s["weights"].shape), "key_cache": None,
            "value_cache": None}


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"summary": _exact_summary, "sparse": _exact_rows, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](case, s)
