"""Float64 oracle of the Q/K preparation and of attention over blocks chosen for each query.

Plain numpy, one query at a time, from the definitions in include/svg.h.  Inputs are float arrays that hold the
values of the device tensors (bf16 or fp32), so nothing here rounds.  The bounds that come with a result say how far
a kernel may be from it whose matrix products take bf16 operands (half a step is 2^-8 of a value) and sum in fp32.
"""
from __future__ import annotations

import numpy as np

HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24


def rotate(x, cos, sin, interleaved: bool):
    """x [..., D] turned by angles [..., D/2]."""
    y = np.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else np.split(x, 2, -1)
    ya, yb = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        y[..., 0::2], y[..., 1::2] = ya, yb
    else:
        y[..., : x.shape[-1] // 2], y[..., x.shape[-1] // 2:] = ya, yb
    return y


def norm_rope(x, w, cos, sin, eps: float, interleaved: bool, pos):
    """x [B, N, H, D], pos [B, N] (negative: padding) -> head-major [B, H, N, D], zeros for padding; and the size of
    each pair (what a rotation's rounding is relative to)."""
    x = np.asarray(x, np.float64)
    B, N, H, D = x.shape
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        n = n * np.asarray(w, np.float64)
    size = np.abs(n)
    if cos is not None:
        at = np.maximum(pos, 0)
        c, s = np.asarray(cos, np.float64)[at][:, :, None], np.asarray(sin, np.float64)[at][:, :, None]
        size = rotate(size, np.abs(c), -np.abs(s), interleaved) + rotate(size, np.abs(c), np.abs(s), interleaved)
        n = rotate(n, c, s, interleaved)
    keep = (pos >= 0)[:, :, None, None]
    return (n * keep).transpose(0, 2, 1, 3), (np.abs(size) * keep).transpose(0, 2, 1, 3)


def norm_rope_backward(x, w, cos, sin, eps: float, interleaved: bool, pos, dy):
    """dy [B, H, N, D] -> (dx [B, N, H, D], dw [D], size of dx's terms, sum of dw's absolute terms)."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    u = np.asarray(dy, np.float64).transpose(0, 2, 1, 3)
    if cos is not None:
        at = np.maximum(pos, 0)
        u = rotate(u, np.asarray(cos, np.float64)[at][:, :, None], -np.asarray(sin, np.float64)[at][:, :, None],
                   interleaved)
    u = u * (pos >= 0)[:, :, None, None]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    g = u if w is None else u * np.asarray(w, np.float64)
    dx = r * (g - n * (g * n).mean(-1, keepdims=True))
    size = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True))
    return dx, (u * n).reshape(-1, D).sum(0), size, np.abs(u * n).reshape(-1, D).sum(0)


def block_means(k, block: int, lens):
    """k [BHk, Nk, D] -> fp32 [BHk, ceil(Nk/block), D]; lens: keys in use of every head."""
    BHk, Nk, D = k.shape
    out = np.zeros((BHk, -(-Nk // block), D), np.float32)
    for h in range(BHk):
        for j in range(-(-lens[h] // block)):
            rows = k[h, j * block:min((j + 1) * block, lens[h])].astype(np.float64)
            out[h, j] = (rows.sum(0) / len(rows)).astype(np.float32)
    return out


def seen_keys(length: int, Nq: int, n: int, causal: bool) -> int:
    return max(0, min(length - Nq + n + 1, length)) if causal else length


def select_blocks(q, mean, block: int, topk: int, sink: int, local: int, causal: bool, lens):
    """q [BHq, Nq, D], mean [BHk, nblk, D] -> [BHk, Nq, topk] int32."""
    BHk, G, Nq = mean.shape[0], q.shape[0] // mean.shape[0], q.shape[1]
    out = np.full((BHk, Nq, topk), -1, np.int32)
    for h in range(BHk):
        m = mean[h].astype(np.float64)
        for n in range(Nq):
            seen = seen_keys(lens[h], Nq, n, causal)
            may = -(-seen // block)
            pos = lens[h] - Nq + n
            mine = pos // block if pos >= 0 else -1
            taken = {j for j in range(may) if j < sink or mine - local < j <= mine}
            score = (q[h * G:(h + 1) * G, n].astype(np.float64).sum(0) * m[:may]).sum(-1)
            score = np.where(np.isnan(score), -np.inf, score)
            rest = sorted((j for j in range(may) if j not in taken), key=lambda j: (-score[j], j))
            chosen = sorted(taken | set(rest[:topk - len(taken)]))
            out[h, n, :len(chosen)] = chosen
    return out


def key_mask(sel, block: int, causal: bool, lens, Nk: int):
    """[BHk, Nq, Nk] bool: the keys a query attends (ids outside the buffer passed over)."""
    BHk, Nq, _ = sel.shape
    nblk = -(-Nk // block)
    mask = np.zeros((BHk, Nq, Nk), bool)
    for h in range(BHk):
        for n in range(Nq):
            seen = seen_keys(lens[h], Nq, n, causal)
            for j in sel[h, n]:
                if 0 <= j < nblk:
                    mask[h, n, j * block:min((j + 1) * block, seen)] = True
    return mask


def attention(q, k, v, sel, block: int, causal: bool, lens, scale: float):
    """(o, lse, bound of o, bound of lse): o [BHq, Nq, D], lse [BHq, Nq]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    BHq, Nq, D = q.shape
    G = BHq // k.shape[0]
    mask = key_mask(sel, block, causal, lens, k.shape[1])
    o, lse = np.zeros_like(q), np.full((BHq, Nq), -np.inf)
    bo, bl = np.zeros_like(q), np.zeros((BHq, Nq))
    for h in range(BHq):
        for n in range(Nq):
            at = np.flatnonzero(mask[h // G, n])
            if len(at) == 0:
                continue
            kk, vv = k[h // G, at], v[h // G, at]
            s = kk @ q[h, n] * scale
            top = s.max()
            p = np.exp(s - top)
            lse[h, n] = top + np.log(p.sum())
            p /= p.sum()
            o[h, n] = p @ vv
            # a score is a sum of D fp32 products
            es = D * HALF_F32 * scale * (np.abs(kk) @ np.abs(q[h, n])).max() + 4 * HALF_F32 * (1 + np.abs(s).max())
            size = p @ np.abs(vv)
            bo[h, n] = HALF_BF16 * np.abs(o[h, n]) + (HALF_BF16 * 1.01 + 2 * es + len(at) * HALF_F32) * size
            bl[h, n] = es + 2.0 ** -20 * (1 + abs(lse[h, n]))
    return o, lse, bo, bl


def attention_backward(do, q, k, v, o, lse, sel, block: int, causal: bool, lens, scale: float):
    """((dq, dk, dv), their bounds) of the given o and lse."""
    do, q, k, v, o = (np.asarray(x, np.float64) for x in (do, q, k, v, o))
    BHq, Nq, D = q.shape
    G = BHq // k.shape[0]
    mask = key_mask(sel, block, causal, lens, k.shape[1])
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(BHq):
        for n in range(Nq):
            at = np.flatnonzero(mask[h // G, n])
            if len(at) == 0:
                continue
            kk, vv = k[h // G, at], v[h // G, at]
            s = kk @ q[h, n] * scale
            p = np.exp(s - float(lse[h, n]))
            dp, delta = vv @ do[h, n], do[h, n] @ o[h, n]
            ds = p * (dp - delta)
            dq[h, n] = scale * (ds @ kk)
            dk[h // G, at] += scale * np.outer(ds, q[h, n])
            dv[h // G, at] += np.outer(p, do[h, n])
            es = D * HALF_F32 * scale * (np.abs(kk) @ np.abs(q[h, n])).max() + 8 * HALF_F32 * (1 + np.abs(s).max())
            ed = D * HALF_F32 * (np.abs(vv) @ np.abs(do[h, n]) + np.abs(do[h, n]) @ np.abs(o[h, n]))
            eds = (HALF_BF16 * 1.01 + 2 * es) * np.abs(ds) + 2 * p * ed
            ep = (HALF_BF16 * 1.01 + 2 * es) * p
            bq[h, n] = scale * (eds @ np.abs(kk))
            bk[h // G, at] += scale * np.outer(eds, np.abs(q[h, n]))
            bv[h // G, at] += np.outer(ep, np.abs(do[h, n]))
    bounds = [b * (1 + Nq * G * HALF_F32) + HALF_BF16 * np.abs(x) * 1.01 + 1e-30
              for b, x in ((bq, dq), (bk, dk), (bv, dv))]
    return (dq, dk, dv), bounds
