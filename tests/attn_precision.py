"""Inputs of attn_decode whose result hangs on bits that a looser check would not see,
with their results in 64 bits and bounds on the error.  numpy only.

scale is ln 2 rounded to binary32 (SCALE): its product with log2(e), which takes scores
to units of log 2, rounds to 1, so such scores are the plain products q.k.  Where those
are exact, so is every exponent, and what is left (u = 2^-24) is: the exponential, 2^-22
= 4u; the weights' parts over 16-bit caches, 2^-22 = 4u; a sum's roundings, u an addition
(2u where the matrix instructions truncate it); the division, 4u with its operands."""
import math

import numpy as np

U = 2.0 ** -24
SCALE = float(np.float32(math.log(2.0)))


def to_f16(x):
    return x.astype(np.float16).astype(np.float64)


def to_bf16(x):
    """Rounded to 8 bits, ties to even (no overflow here)."""
    b = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7fff + (b >> 16 & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def exact(q, k, v):
    """q [rows][heads][D] on one K/V head's k, v [rows][n][D]: out, and the weights
    [rows][heads][n]; scores in units of log 2."""
    s = np.einsum("mgd,mnd->mgn", q, k)
    p = np.exp2(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return np.einsum("mgn,mnd->mgd", p, v), p


LEVELS = (4, 8, 10, 12, 16, 20, 32, 50)


def small_weights(heads, dim, n, at):
    """Row m: one entry in 16, `at` the first, has all of the weight but 2^-LEVELS[m] to
    2^-1.9 LEVELS[m] (by the head), and no value: out is made of the small weights alone."""
    rows = len(LEVELS)
    q, k = np.zeros((rows, heads, dim)), np.zeros((rows, n, dim))
    q[:, :, 0] = 1 + np.arange(heads) % 8 / 8
    k[:, :, 0] = -0.375
    k[:, at::16, 0] = np.array(LEVELS)[:, None]
    v = 1 + np.random.default_rng(dim + n).integers(0, 128, (rows, n, dim)) / 128
    v[:, at::16] = 0
    return q, k, v


def small_weights_bound(want, n):
    # positive terms: the exponential and the parts, n truncated additions, the division
    return (4 + 4 + 2 * n + 4 + n + 4) * U * want


def small_values_of_q(heads, dim):
    """A first value of 2^12 that meets keys of 0 (it sets what a head's q is measured by), the
    others some 2^-14, that meet keys of 2^15 one by one: scores of 2 to 4.  V: the unit matrix."""
    r = np.random.default_rng(dim + 1)
    q = 2.0 ** -14 * (1 + r.integers(0, 1 << 23, (1, heads, dim)) * 2.0 ** -23)
    q[:, :, 0] = 2.0 ** 12
    k, v = np.zeros((1, dim - 1, dim)), np.zeros((1, dim - 1, dim))
    i = np.arange(dim - 1)
    k[0, i, i + 1], v[0, i, i] = 2.0 ** 15, 1
    return q, k, v


def small_values_of_q_bound(want, dim):
    # scores of at most 4 off by 2^-22 (q's parts) and u (a difference), ln2 each
    return (2 * (16 * U + 4 * U + 8 * U) + (3 * dim + 8) * U) * want
