"""Plain forms of the quantised K/V caches' operators in numpy, from their definitions:
rounded where the formats round, in 64 bits elsewhere."""
import numpy as np

import decode_ref as ref

U = ref.U32
F32, F16 = np.float32, np.float16
KINDS = ("i8", "u4")


def half_away(x):
    """x (binary32) to the nearest integer, halves away from zero."""
    t = np.trunc(x)
    return t + np.copysign((np.abs(x - t) >= 0.5).astype(F32), x)


def quantise(x, kind):
    """x [..., D] binary32: codes [..., D] and the blocks' words [..., D / 32] (i8) or [..., D / 32, 2]."""
    x = np.asarray(x, dtype=F32)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    fine = np.isfinite(b).all(-1)
    z = np.where(fine[..., None], b, F32(0))
    with np.errstate(all="ignore"):
        if kind == "i8":
            d = np.abs(z).max(-1) / F32(127)
            q = np.where(d[..., None] == 0, F32(0), half_away(z / d[..., None]))
            q = np.clip(np.where(np.isfinite(q), q, 0), -127, 127)
            return q.reshape(x.shape).astype(np.int8), np.where(fine, d, F32(np.nan))
        lo = z.min(-1)
        s = ((z.max(-1) - lo) / F32(15)).astype(F16)
        m = lo.astype(F16)
        fine &= np.isfinite(s) & np.isfinite(m)
        q = half_away((z - m.astype(F32)[..., None]) / s.astype(F32)[..., None])
        q = np.where((fine & (s != 0))[..., None], np.clip(np.nan_to_num(q), 0, 15), 0)
    words = np.stack((np.where(fine, s, F16(np.nan)), np.where(fine, m, F16(np.nan))), -1)
    return q.reshape(x.shape).astype(np.uint8), words


def pack(codes, kind):
    return codes if kind == "i8" else codes[..., 0::2] | codes[..., 1::2] << 4


def unpack(codes, kind):
    return codes if kind == "i8" else np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))


def values(packed, words, kind, spread=False):
    """The values [..., D] in 64 bits; spread: the sum of the magnitudes that they are made of, where
    a u4 value may be m and s code, or m + 15 s and s (15 - code) (half of an output's entries are: codes
    have no sign, and truncated sums of all would lean one way)."""
    q = unpack(packed, kind).astype(np.float64)
    q = q.reshape(q.shape[:-1] + (-1, 32))
    if kind == "i8":
        v = q * words.astype(np.float64)[..., None]
        v = np.abs(v) if spread else v
    else:
        s, m = words[..., 0:1].astype(np.float64), words[..., 1:2].astype(np.float64)
        v = np.maximum(np.abs(m) + s * q, np.abs(m + 15 * s) + s * (15 - q)) if spread else m + s * q
    return v.reshape(v.shape[:-2] + (-1,))


def entry_major(v):
    """[rows][kv_heads][n][D] as attn_decode's [rows][n][kv_heads * D]."""
    rows, h, n, d = v.shape
    return v.transpose(0, 2, 1, 3).reshape(rows, n, h * d)


def attn(q, k, v, k_spread, v_spread, pos, heads, window, sinks, scale, acc=None):
    """q [rows][heads * D], values [rows][kv_heads][n_pos][D]: out, its bound, acc and its bound.

    The bounds, u = 2^-24.  A score is a sum over blocks of s (or d) times a sum of products,
    and of m times a sum of q: exact products of parts that hold 22 bits of q (4u), at most D
    of them truncated where the matrix instructions add them (2u each, of the largest term or
    partial sum), four roundings a block and the sums of q (32 + 4 of u), so
    |ds| <= (2D + 64) u sum|q| (s code + |m|) scale.  A weight carries 2 |ds| and 8u (the
    exponential, its argument's rounding, the reference), its product with a block's scale and
    its three exact parts u, n entries' sums 2n u (truncated), and so does the normalising sum."""
    rows, kv_heads, n_pos, dim = k.shape
    group = heads // kv_heads
    out, tol = np.zeros((rows, heads * dim)), np.zeros((rows, heads * dim))
    new_acc = None if acc is None else acc.astype(np.float64).copy()
    acc_tol = None if acc is None else np.zeros_like(new_acc)
    for m in range(rows):
        see = ref.visible(int(pos[m]), window, sinks)
        if not see:
            continue
        n = len(see)
        for h in range(kv_heads):
            kk, vv, ka, va = (x[m, h][see] for x in (k, v, k_spread, v_spread))
            for g in range(h * group, (h + 1) * group):
                cols = slice(g * dim, (g + 1) * dim)
                qq = q[m, cols]
                s = kk @ qq * scale
                e = np.exp(s - s.max())
                p = e / e.sum()
                ds = (2 * dim + 64) * U * float((ka @ np.abs(qq)).max()) * abs(scale)
                rel = 2 * (2 * ds + 10 * U + 2 * n * U)
                out[m, cols] = p @ vv
                tol[m, cols] = rel * (p @ va)
                if acc is not None:
                    new_acc[m, h, see] += p
                    acc_tol[m, h, see] += rel * p
    if acc is not None:   # the sum itself: one rounding a head and one into acc
        acc_tol += (group + 1) * U * np.abs(new_acc)
    return out, tol, new_acc, acc_tol


def evict(planes, pos, acc, budget, sinks, recent):
    """planes [rows][kv_heads][n_pos][...]: the new planes, pos, acc and kept."""
    rows, kv_heads, n_pos = acc.shape
    index = np.broadcast_to(np.arange(n_pos)[None, :, None], (rows, n_pos, kv_heads))
    old, _, new_pos, new_acc, kept = ref.evict(np.ascontiguousarray(index), np.zeros((rows, n_pos, kv_heads)), pos, acc,
                                               kv_heads, budget, sinks, recent, n_pos)
    planes = [p.copy() for p in planes]
    for p in planes:
        for m in range(rows):
            for h in range(kv_heads):
                p[m, h] = p[m, h][old[m, :, h]]
    return planes, new_pos, new_acc, kept
