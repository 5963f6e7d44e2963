"""Plain 64-bit forms of the decode step's operators around the projections
(attention over the caches, eviction, sampling), row by row in numpy, written
from the operators' definitions."""
import math

import numpy as np

U32 = 2.0 ** -24   # half a step of binary32, relative


def visible(pos, window, sinks):
    n = pos + 1
    return [i for i in range(n) if window < 0 or i < sinks or i >= n - window]


def attn(q, k, v, pos, heads, kv_heads, window, sinks, scale, acc=None):
    """q [rows][heads*D], caches [rows][n_pos][kv_heads*D], all float64.
    Returns out, the new acc (or None) and bounds on a binary32 evaluation's
    errors of both.

    The bounds, with u = 2^-24: a score is a sum of D products, each operand
    rounded at most once more (the scale): |ds| <= (D + 4) u sum|q k| scale.
    A weight exp(s - m) then carries a relative 2 |ds|max + 8u (the maximum's
    own error included; the exponential and the steps around it a few u), its
    sums over n entries n u more, and the same again for the normalising sum.
    (Operands carried as two or three 16-bit parts hold 22 bits at least: 4u of a
    score's product and 4u of a weight, within the D + 4 and the 8.)"""
    rows, n_pos, _ = k.shape
    dim = k.shape[2] // kv_heads
    group = heads // kv_heads
    out = np.zeros((rows, heads * dim))
    tol = np.zeros_like(out)
    new_acc = None if acc is None else acc.astype(np.float64).copy()
    acc_tol = None if acc is None else np.zeros_like(new_acc)
    for m in range(rows):
        see = visible(int(pos[m]), window, sinks)
        if not see:
            continue
        n = len(see)
        for g in range(heads):
            h = g // group
            kk, vv = k[m, see, h * dim:(h + 1) * dim], v[m, see, h * dim:(h + 1) * dim]
            qq = q[m, g * dim:(g + 1) * dim]
            s = kk @ qq * scale
            e = np.exp(s - s.max())
            p = e / e.sum()
            ds = (dim + 4) * U32 * float((np.abs(kk) @ np.abs(qq)).max()) * abs(scale)
            rel = 2 * (2 * ds + 8 * U32 + n * U32)
            out[m, g * dim:(g + 1) * dim] = p @ vv
            tol[m, g * dim:(g + 1) * dim] = rel * (p @ np.abs(vv))
            if acc is not None:
                new_acc[m, h, see] += p
                acc_tol[m, h, see] += rel * p
    if acc is not None:   # the sum itself: one rounding a head and one into acc
        acc_tol += (group + 1) * U32 * np.abs(new_acc)
    return out, tol, new_acc, acc_tol


def evict(k, v, pos, acc, kv_heads, budget, sinks, recent, n_pos):
    """Returns new k, v, pos, acc and kept, as written (copies of the inputs'
    own type)."""
    k, v, acc, old = k.copy(), v.copy(), acc.copy(), acc
    rows, dim = k.shape[0], k.shape[2] // kv_heads
    new_pos = np.array(pos, dtype=np.int32)
    kept = np.full((rows, kv_heads, budget), -1, dtype=np.int32)
    for m in range(rows):
        n = int(pos[m]) + 1
        if n < 0 or n > n_pos:
            continue
        for h in range(kv_heads):
            if n <= budget:
                kept[m, h, :n] = np.arange(n)
                continue
            # sort by weight, the largest first, NaN last; ties by index
            mid = sorted(range(sinks, n - recent),
                         key=lambda i: (math.isnan(old[m, h, i]), -old[m, h, i] if not math.isnan(old[m, h, i]) else 0, i))
            idx = sorted(list(range(sinks)) + mid[:budget - sinks - recent] + list(range(n - recent, n)))
            cols = slice(h * dim, (h + 1) * dim)
            k[m, :budget, cols] = k[m, idx, cols].copy()
            v[m, :budget, cols] = v[m, idx, cols].copy()
            acc[m, h] = 0
            acc[m, h, :budget] = old[m, h, idx]
            kept[m, h] = idx
            new_pos[m] = budget - 1
    return k, v, new_pos, acc, kept


def sample(x, u, t=1.0, k=0, p=1.0, mp=0.0):
    """(token, probability, kept) of one row, in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    ids = [i for i in range(len(x)) if x[i] > -math.inf]
    if not ids or not t >= 0 or math.isnan(p) or math.isnan(mp):
        return 0, 0.0, 0
    ids.sort(key=lambda i: (-x[i], i))
    if t < 2.0 ** -60:
        return ids[0], 1.0, 1
    top = x[ids[0]]
    w = {i: 1.0 if x[i] == top else 0.0 if top == math.inf else math.exp((x[i] - top) / t) for i in ids}
    if k > 0:
        ids = ids[:k]
    if p < 1:
        mass, goal, end = 0.0, float(p) * math.fsum(w[i] for i in ids), 0
        for end, i in enumerate(ids):
            mass += w[i]
            if mass >= goal:
                break
        ids = ids[:end + 1]
    ids = [i for j, i in enumerate(ids) if j == 0 or w[i] >= mp]
    total, cdf = math.fsum(w[i] for i in ids), 0.0
    tok = None
    for i in sorted(ids):
        cdf += w[i]
        if w[i]:
            tok = i
        if cdf > (u if u > 0 else 0.0) * total:
            break
    return tok, w[tok] / total, len(ids)
