"""Plain definitions of the operators that read or keep a long context in part, one
block and one token at a time.  Nothing here uses the library.

Bounds and scores are whole numbers and single fp32 operations, so they are computed
exactly and compared for equality."""
import numpy as np
import torch

F = np.float32


def values(pool):
    """Keys as the values their codes stand for, without a pool's scale."""
    if pool.dtype == torch.uint8:
        pool = pool.cpu().view(torch.float8_e4m3fn)
    return pool.float().cpu().numpy()


def code(x):
    """(int codes, fp32 scale) of one vector set with a common amplitude."""
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(x).max() if x.size else F(0)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, dtype=np.int64), F(np.inf)
    if top < F(2.0 ** -40):
        return np.zeros(x.shape, dtype=np.int64), F(0)
    inv = F(127) / F(top)
    return np.rint(x.astype(F) * inv).astype(np.int64), F(top) * (F(1) / F(127))


def summarize(codes, scales, keys, tables, ctx, start=None):
    """codes int8 [N, K, 2, D] and scales [N, K] (numpy, changed in place)."""
    bs = keys.shape[1]
    for s, c in enumerate(ctx):
        n = c if start is None else start[s + 1] - start[s]
        for j in range((c - n) // bs, -(-c // bs)) if n > 0 else ():
            b = tables[s][j]
            for h in range(keys.shape[2]):
                k = keys[b, :min(bs, c - j * bs), h]
                bad = not np.isfinite(k).all()
                lo_hi = np.stack([k.min(0), k.max(0)]) if not bad else np.full((2, k.shape[1]),
                                                                              np.nan)
                codes[b, h], scales[b, h] = code(lo_hi)


def scores(query, codes, scales, table, have, kh, group):
    """fp32 scores of the `have` blocks of a table row for one KV head."""
    out = np.zeros(have, dtype=F)
    q = [code(query[h].astype(F)) for h in range(kh * group, (kh + 1) * group)]
    for j in range(have):
        b = table[j]
        if np.isposinf(scales[b, kh]):
            out[j] = np.inf
            continue
        best = None
        for c, s in q:
            s = F(0) if np.isinf(s) else s
            total = np.maximum(c * codes[b, kh, 0].astype(np.int64),
                               c * codes[b, kh, 1].astype(np.int64)).sum()
            with np.errstate(over="ignore"):
                x = F(s) * F(total)
            best = x if best is None else max(best, x)
        with np.errstate(over="ignore"):
            out[j] = best * F(scales[b, kh])
    return out


def select(query, codes, scales, tables, seq, pos, bs, top_k, first, last, kv_heads):
    """int32 [T, K, top_k]; query a float numpy array [T, H, D]."""
    T, H, _ = query.shape
    out = np.full((T, kv_heads, top_k), -1, dtype=np.int32)
    for t in range(T):
        if seq[t] < 0:
            continue
        have = pos[t] // bs + 1
        for h in range(kv_heads):
            if have <= top_k:
                out[t, h, :have] = np.arange(have)
                continue
            x = scores(query[t], codes, scales, tables[seq[t]], have, h, H // kv_heads)
            mid = np.arange(first, have - last)
            best = mid[np.lexsort((mid, -x[mid].astype(np.float64)))][:top_k - first - last]
            out[t, h] = np.sort(np.concatenate([np.arange(first), best,
                                                np.arange(have - last, have)]))
    return out


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # eps / 2


def attend(q, k, v, scale, out_dtype, p_dtype):
    """One query vector over keys and values [n, D] in 64 bits: (output, its tolerance,
    weights, theirs).  Counted: the output's half step; the weights' half step as a
    matrix operand, which moves the output by at most that times sum w |v|; a score's
    fp32 error, which moves its own weight and the sum of weights; the sums' own."""
    x = k @ q * scale
    with np.errstate(invalid="ignore"):
        w = np.exp(x - x.max())
    w /= w.sum()
    o = w @ v
    size = scale * (np.abs(k) @ np.abs(q)).max()
    e = 2 * ((len(q) + 4) * 2.0 ** -22 * size + (len(x) + 8) * 2.0 ** -23)
    tol = HALF_STEP[out_dtype] * np.abs(o) + \
        1.01 * (HALF_STEP[p_dtype] + e) * (w @ np.abs(v)) + 2.0 ** -24
    return o, tol, w, w * e


def pool_values(pool, scale):
    if pool.dtype == torch.uint8:
        return pool.cpu().view(torch.float8_e4m3fn).double().numpy() * scale
    return pool.double().cpu().numpy()


def sparse_attention(q, kc, vc, tables, seq, pos, chosen, scale, out_dtype, p_dtype):
    """(output, tolerance) of every row over the blocks of its lists (int arrays, negative
    entries left out); kc and vc are pools of values in 64 bits."""
    q = q.double().cpu().numpy()
    T, H, D = q.shape
    bs, K = kc.shape[1:3]
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    for t in range(T):
        if seq[t] < 0:
            continue
        for h in range(K):
            blk = chosen[t][h][:min(len(chosen[t][h]), pos[t] // bs + 1)]
            p = np.concatenate([np.arange(b * bs, b * bs + bs) for b in blk if b >= 0] +
                               [np.zeros(0, dtype=int)]).astype(int)
            p = p[p <= pos[t]]
            if not len(p):
                continue
            at = tables[seq[t]][p // bs]
            for g in range(h * H // K, (h + 1) * H // K):
                out[t, g], tol[t, g], _, _ = attend(q[t, g], kc[at, p % bs, h], vc[at, p % bs, h],
                                                    scale, out_dtype, p_dtype)
    return out, tol


def weights_attention(q, kc, vc, weights, tables, ctx, weighted, scale, out_dtype, p_dtype):
    """(output, tolerance, weights_out, tolerance) of a decode step; entries of weights
    that no context reaches come back as they are, with a tolerance of 0."""
    q = q.double().cpu().numpy()
    S, H, D = q.shape
    bs, K = kc.shape[1:3]
    out, tol = np.zeros((S, H, D)), np.zeros((S, H, D))
    new, new_tol = weights.astype(np.float64).copy(), np.zeros(weights.shape)
    for s in range(S):
        p = np.arange(ctx[s])
        at, row = tables[s][p // bs], p % bs
        total, err = np.zeros(len(p)), np.zeros(len(p))
        for h in range(K):
            for g in range(h * H // K, (h + 1) * H // K) if len(p) else ():
                out[s, g], tol[s, g], w, e = attend(q[s, g], kc[at, row, h], vc[at, row, h],
                                                    scale, out_dtype, p_dtype)
                total, err = total + w, err + e
        before = np.where(p < weighted[s], new[at, row], 0.0) if len(p) else total
        new[at, row] = before + total
        # H terms added one by one, then the sum so far
        new_tol[at, row] = err + (H + 8) * 2.0 ** -24 * total + \
            2.0 ** -24 * (before + total) + 2.0 ** -40
    return out, tol, new, new_tol


def plan_eviction(tables, ctx, weights, free, count, bs, limit, budget, sinks, recent, capacity):
    """(moves [S, capacity, 2], lengths, free, count, weights) by the definition; None for
    a plan that is refused.  numpy arrays, none of them changed."""
    free, out = free.copy(), weights.copy()
    N = len(free)
    moves = np.full((len(ctx), capacity, 2), -1, dtype=np.int32)
    end = np.asarray(ctx).copy()
    for s, c in enumerate(ctx):
        if c <= limit:
            continue
        end[s] = budget
        slot = np.array([int(tables[s][p // bs]) * bs + p % bs for p in range(c)])
        ranked = sorted(range(sinks, c - recent),
                        key=lambda p: (-(weights.flat[slot[p]] if weights.flat[slot[p]] > 0
                                         else 0.0), p))
        gone = set(ranked[budget - sinks - recent:])
        late = [p for p in range(budget, c) if p not in gone]
        holes = [p for p in range(budget) if p in gone]
        assert len(late) == len(holes)
        for i, (a, b) in enumerate(zip(late, holes)):
            moves[s, i] = slot[a], slot[b]
            out.flat[slot[b]] = weights.flat[slot[a]]
        for j in range(-(-budget // bs), -(-c // bs)):
            if count >= N:
                return None
            free[count] = tables[s][j]
            count += 1
    return moves, end, free, count, out
