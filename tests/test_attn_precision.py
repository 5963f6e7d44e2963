"""The precision checks of attn_decode find what they are there to find: arithmetic of
fewer bits, and parts of a row that are lost, fall outside their bounds (CPU, numpy)."""
import numpy as np
import pytest

import attn_precision as ap

rng = np.random.default_rng


def out_of(p, v, w):
    """out from weights w (of any precision) over the sum of exact ones p."""
    return np.einsum("mgn,mnd->mgd", w, v) / p.sum(-1)[..., None]


def unscaled(q, k):
    s = np.einsum("mgd,mnd->mgn", q, k)
    return np.exp2(s - s.max(-1, keepdims=True))


def two_parts(x, to):
    hi = to(x)
    return hi + to(x - hi)


def test_scale_takes_scores_to_units_of_log_2():
    assert np.float32(float(np.float32(ap.SCALE)) * 1.4426950408889634) == 1.0


@pytest.mark.parametrize("n,at", [(16, 0), (300, 5)])
def test_small_weights_need_more_than_two_parts_of_f16(n, at):
    q, k, v = ap.small_weights(8, 64, n, at)
    want, _ = ap.exact(q, k, v)
    p, tol = unscaled(q, k), ap.small_weights_bound(want, n)
    got = out_of(p, v, two_parts(p * 128, ap.to_f16) / 128)        # 22 bits of the largest weights only
    bad = (np.abs(got - want) > tol).any(axis=(1, 2))
    assert bad[3:].all()                                            # from 2^-12 to 2^-24 on
    hi = p * 128
    lo = ap.to_f16((hi - ap.to_f16(hi)) * 2048) / 2048              # the second part 2^11 lower
    assert (np.abs(out_of(p, v, (ap.to_f16(hi) + lo) / 128) - want) > tol).any()
    assert np.all(np.abs(out_of(p, v, p.astype(np.float32).astype(np.float64)) - want) <= tol)


@pytest.mark.parametrize("n", [64, 600])
def test_cancelling_weights_need_18_bits(n):
    q, k, v = ap.cancelling_weights(8, 64, n)
    want, _ = ap.exact(q, k, v)
    p, tol = unscaled(q, k), ap.cancelling_weights_bound(want, n)
    for w in (ap.to_bf16(p), two_parts(p, ap.to_bf16), ap.to_f16(p)):
        assert (np.abs(out_of(p, v, w) - want) > tol).any(-1).all()             # in every head
    assert np.all(np.abs(out_of(p, v, p.astype(np.float32).astype(np.float64)) - want) <= tol)


@pytest.mark.parametrize("dim", [64, 80, 200, 256])
def test_scores_need_the_low_parts_of_q(dim):
    for kv, to in (("bf16", ap.to_bf16), ("f16", ap.to_f16)):
        q, k, v = ap.low_parts_of_q(kv, 8, dim)
        assert np.array_equal(q, q.astype(np.float32))
        want, _ = ap.exact(q, k, v)
        tol = ap.low_parts_of_q_bound(want, kv, 8, dim)
        less = [to(q)] if kv == "f16" else [to(q), two_parts(q, to)]
        if kv == "bf16":          # one step of 16 values without its third part, or with its neighbour's
            low = q - two_parts(q, to)
            for step in range((dim + 15) // 16):
                other = low.copy()
                other[:, :, 16 * step:16 * step + 16] = 0
                less.append(two_parts(q, to) + other)
        for x in less:
            assert (np.abs(ap.exact(x, k, v)[0] - want) > tol).any(-1).all()


@pytest.mark.parametrize("dim", [64, 80, 256])
def test_scores_need_the_small_values_of_q(dim):
    q, k, v = ap.small_values_of_q(8, dim)
    want, _ = ap.exact(q, k, v)
    tol = ap.small_values_of_q_bound(want, dim)
    x = two_parts(q * 2, ap.to_f16) / 2                    # (brought to 2^13)
    assert (np.abs(ap.exact(x, k, v)[0] - want) > tol).any(-1).all()
    hi = ap.to_f16(q * 2)
    x = (hi + ap.to_f16((q * 2 - hi) * 2048) / 2048) / 2   # the second part 2^11 lower
    assert np.all(np.abs(ap.exact(x, k, v)[0] - want) <= tol)


@pytest.mark.parametrize("heads,dim,n", [(1, 64, 60000), (1, 8, 70000), (3, 24, 60000), (1, 256, 40000), (8, 128, 30000)])
def test_a_part_lost_from_a_long_row_is_seen(heads, dim, n):
    """Any of 304 parts (two CTAs an SM) that the join of values leaves out, or weighs 1% wrong
    where a column has few of them."""
    r = rng(dim + n)
    q, k = r.standard_normal((heads, dim)), r.standard_normal((n, dim))
    v = ap.sliced_values(n, dim)
    _, p = ap.exact(q[None] * dim ** -0.5 / ap.SCALE, k[None], v[None])
    want = p[0] @ v
    tol = ap.long_row_bound(q, k, want, dim ** -0.5)
    for part in range(0, 304, 7):
        a, b = n * part // 304, n * (part + 1) // 304
        lost = p[0][:, a:b] @ v[a:b]
        assert (lost > 4 * tol).any(-1).all()
        if dim >= 64:
            assert (0.01 * lost > tol).any(-1).all()
