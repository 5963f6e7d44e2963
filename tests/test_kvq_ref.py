"""The quantised caches' formats: the plain form against the CPU oracle, and what it loses."""
import numpy as np
import pytest

import kvq_ref as kr


def test_i8_is_the_one_word_activation_code(orc):
    x = np.random.default_rng(0).standard_normal((50, 128)).astype(np.float32) * 3
    x[3] = 0
    q, d = orc.act_quant_i8(x)
    codes, words = kr.quantise(x, "i8")
    assert np.array_equal(codes, np.asarray(q).reshape(50, 128)) and np.array_equal(words, np.asarray(d).reshape(50, 4))


@pytest.mark.parametrize("kind", kr.KINDS)
def test_values_are_within_half_a_step(kind):
    x = (np.random.default_rng(1).standard_normal((200, 64)) + 0.7).astype(np.float32)
    codes, words = kr.quantise(x, kind)
    v = kr.values(kr.pack(codes, kind), words, kind)
    b = x.reshape(200, 2, 32).astype(np.float64)
    if kind == "i8":
        step = np.abs(b).max(-1) / 127
        slack = 0
    else:
        step = (b.max(-1) - b.min(-1)) / 15
        # s and m are off by 2^-11 of themselves: 15 steps of s, and m
        slack = 15 * step * 2.0 ** -11 + np.abs(b.min(-1)) * 2.0 ** -11
    off = np.abs(v - x).reshape(200, 2, 32).max(-1)
    assert np.all(off <= step * (0.5 + 1e-4) + slack)


def test_packing_keeps_codes():
    codes = np.random.default_rng(2).integers(0, 16, (3, 5, 96)).astype(np.uint8)
    packed = kr.pack(codes, "u4")
    assert packed.shape == (3, 5, 48) and np.array_equal(kr.unpack(packed, "u4"), codes)
    assert packed[0, 0, 1] == codes[0, 0, 2] + 16 * codes[0, 0, 3]


@pytest.mark.parametrize("kind", kr.KINDS)
def test_blocks_that_cannot_be_held_are_nan(kind):
    x = np.ones((5, 32), dtype=np.float32)
    x[0, 3], x[1, 31], x[2, 0] = np.nan, np.inf, -np.inf
    x[3, 5] = 3e38                       # (binary16 has no such scale)
    codes, words = kr.quantise(x, kind)
    v = kr.values(kr.pack(codes, kind), words, kind)
    assert np.isnan(v[:3]).all() and np.isfinite(v[4]).all()
    assert np.isnan(v[3]).all() == (kind == "u4")
