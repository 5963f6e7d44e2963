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


def cancelling_weights(heads, dim, n):
    """Values of +1 and -1 in turn, weights of 1 and 1 - d in turn (n even), where d is one of
    2^-10 (1 + (2j + 1) 2^-8): 1 - d needs 18 bits, and out is d / (2 - d)."""
    d = 2.0 ** -10 * (1 + (2 * (np.arange(heads) % 8) + 1) * 2.0 ** -8)
    q, k, v = np.zeros((1, heads, dim)), np.zeros((1, n, dim)), np.ones((1, n, dim))
    q[0, :, 1] = (-np.log2(1 - d)).astype(np.float32)
    k[:, 1::2, 1] = -1
    v[:, 1::2] = -1
    return q, k, v


def cancelling_weights_bound(want, n):
    # half of the entries are off by the exponential (4u) and the parts (4u), and a pair's
    # two additions by 2u of its weight, 1: each counts half of that in out; and out's own part
    return 6 * U + (n + 16) * U * np.abs(want)


def low_parts_of_q(kv, heads, dim):
    """Entry i has keys K and -K at values i and i + 1, where q is 1 + m 2^-15 + a 2^-23, with
    m the head's (130 to 186) and |a| <= 64 each value's own: the leading 16 bits cancel, and
    the score is K 2^-23 (a_i - a_i+1) without an error.  V is the unit matrix: out is p."""
    r = np.random.default_rng(dim)
    K = 2.0 ** 15 if kv == "f16" else 2.0 ** 19            # (f16 ends at 2^16)
    m, a = 130 + 8 * (np.arange(heads) % 8), r.integers(-64, 65, (heads, dim))
    q = (1 + m[:, None] * 2.0 ** -15 + a * 2.0 ** -23)[None]
    k, v = np.zeros((1, dim - 1, dim)), np.zeros((1, dim - 1, dim))
    i = np.arange(dim - 1)
    k[0, i, i], k[0, i, i + 1], v[0, i, i] = K, -K, 1
    return q, k, v


def low_parts_of_q_bound(want, kv, heads, dim):
    # scores below 2^3.1 and exact, a difference of two rounded: 16 ln2 u; all of that once
    # more in the sum.  An f16 cache's q holds 22 bits of each value at least when eight
    # heads share it: two values off by 2^-23, times K, ln2.
    ds = 2 * 2.0 ** -23 * 2.0 ** 15 * math.log(2) if kv == "f16" and heads > 4 else 0
    return (2 * (1.01 * ds + 12 * U + 8 * U) + (3 * dim + 8) * U) * want + 2.0 ** -100


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


def sliced_values(n, dim):
    """Values that are 1 in one slice of the n entries a column, 0 elsewhere: a column is its
    slice's weight, and a part of the entries that is lost is a large part of some column."""
    v = np.zeros((n, dim))
    v[np.arange(n), np.arange(n) * dim // n] = 1
    return v


def long_row_bound(q, k, want, scale):
    """Of a column of sliced_values.  A score: (D + 4) u sum |q k| scale at most; a weight and
    the sum of all each carry twice that and the exponential.  Sums of positive terms: the
    roundings of n additions are independent, 8 sqrt(n) u covers more than eight of their
    standard deviations; the matrix instructions' truncation, in chains of 8 at most, 16u."""
    n, dim = k.shape
    ds = (dim + 4) * U * (np.abs(k) @ np.abs(q).T).max(0) * abs(scale)       # [heads]
    return (2 * (2 * ds + 8 * U + 8 * math.sqrt(n) * U + 16 * U))[:, None] * want
