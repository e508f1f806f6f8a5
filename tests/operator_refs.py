"""Plain 64-bit definitions of the serving-step operators and the bounds their
tests hold the kernels to.  Nothing here uses the library."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # eps / 2


def step_maps(tables, ctx, new, free, count, bs, capacity):
    """The step's arrays by the definition, one block and one token at a time
    (numpy int arrays in, a dict out); None for a step that is refused."""
    tables, free = tables.copy(), free.copy()
    S, MB = tables.shape
    N = len(free)
    ctx, new = [int(x) for x in ctx], [int(x) for x in new]
    for c, n in zip(ctx, new):
        if c < 0 or n < -1 or c + max(n, 0) > MB * bs:
            return None
    if sum(max(n, 0) for n in new) > capacity or count < 0:
        return None
    for s in range(S):
        if new[s] == -1:
            for j in range(-(-ctx[s] // bs)):
                if count >= N:
                    return None
                free[count] = tables[s, j]
                count += 1
    out = dict(start=[0], seq=[], pos=[], slot=[], ctx=[])
    for s in range(S):
        if new[s] == -1:
            out["start"].append(out["start"][-1])
            out["ctx"].append(0)
            continue
        for j in range(-(-ctx[s] // bs), -(-(ctx[s] + new[s]) // bs)):
            if count == 0:
                return None
            count -= 1
            tables[s, j] = free[count]
        for p in range(ctx[s], ctx[s] + new[s]):
            out["seq"].append(s)
            out["pos"].append(p)
            out["slot"].append(int(tables[s, p // bs]) * bs + p % bs)
        out["start"].append(out["start"][-1] + new[s])
        out["ctx"].append(ctx[s] + new[s])
    for k in ("seq", "pos", "slot"):
        out[k] += [-1] * (capacity - len(out[k]))
    return dict({k: np.array(v, dtype=np.int32) for k, v in out.items()}, tables=tables,
                free=free, count=count)


def rope(x, pos, inv_freq, axis, interleaved):
    """(rotated x, bound of its fp32 error) for x [T, heads, d], pos [axes, T]."""
    x = x.double().cpu().numpy()
    f = inv_freq.double().cpu().numpy()
    h = len(f)
    phi = np.stack([pos[axis[i]].astype(np.float64) * f[i] for i in range(h)], -1)[:, None, :]
    i, j = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else \
        (np.arange(h), np.arange(h, 2 * h))
    u, v = x[..., i], x[..., j]
    y, err = x.copy(), np.zeros_like(x)
    y[..., i] = u * np.cos(phi) - v * np.sin(phi)
    y[..., j] = v * np.cos(phi) + u * np.sin(phi)
    # the phase in turns: 48 bits of f / 2 pi and three fp32 sums of fractions;
    # sine and cosine to an ulp; two products and a sum
    turns = np.abs(phi) / (2 * math.pi)
    e = 2 * math.pi * (turns * 2.0 ** -45 + 2.0 ** -23) + 2.0 ** -22 + 3 * 2.0 ** -24
    err[..., i] = err[..., j] = (np.abs(u) + np.abs(v)) * e
    return y, err


def pool_values(pool, scale=1.0):
    if pool.dtype == torch.uint8:
        return pool.cpu().view(torch.float8_e4m3fn).double().numpy() * scale
    return pool.double().cpu().numpy()


def visible(pos, n, window, sinks):
    p = np.arange(n)
    return p[(p <= pos) & ((p > pos - window) | (p < sinks))]


def window_attention(q, kc, vc, tables, start, ctx, scale, window, sinks, out_dtype,
                     p_dtype):
    """(output, tolerance) of every row, in 64 bits, from pools of values
    [blocks, bs, Hkv, d].  The tolerance counts the roundings of the kernels:
    the output's half step; the weights' half step as a matrix operand, which
    moves the output by at most that times sum w |v|; fp32 scores and sums."""
    q = q.double().cpu().numpy()
    T, H, D = q.shape
    bs, K = kc.shape[1], kc.shape[2]
    G = H // K
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    for s, c in enumerate(ctx):
        c = int(c)
        lo, hi = int(start[s]), int(start[s + 1])
        for r in range(lo, hi):
            pos = c - (hi - lo) + (r - lo)
            p = visible(pos, c, window, sinks) if pos >= 0 else np.zeros(0, dtype=int)
            if not len(p):
                continue
            blk = tables[s][p // bs]
            for h in range(K):
                k, v = kc[blk, p % bs, h], vc[blk, p % bs, h]
                for g in range(h * G, (h + 1) * G):
                    x = k @ q[r, g] * scale
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    o = w @ v
                    mass = w @ np.abs(v)
                    size = scale * (np.abs(k) @ np.abs(q[r, g])).max()
                    # a score's error moves its weight, and the sum of weights
                    e = 2 * ((D + 4) * 2.0 ** -22 * size + (len(p) + 8) * 2.0 ** -23)
                    out[r, g] = o
                    tol[r, g] = (HALF_STEP[out_dtype] * np.abs(o) +
                                 1.01 * (HALF_STEP[p_dtype] + e) * mass + 2.0 ** -24)
    return out, tol


def assert_within(got, want, tol, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    far = np.abs(got - want)
    over = far > tol
    assert not over.any(), \
        f"{what}: {over.sum()} past their bound, worst {np.max(far[over] / (tol[over] + 1e-300)):.2f}x"
