"""GPU tests of the quantised K/V caches: stored tokens and read-back entries bit for bit,
attention against 64 bits, eviction exactly, and a run of them together."""
import math

import numpy as np
import pytest

import attn_precision as ap
import kvq_ref as kr
from q8_quantized_projection_gb300 import native

pytestmark = pytest.mark.gpu
KINDS = list(kr.KINDS)
FLOATS = ["f32", "f16", "bf16"]


def torch():
    import torch as _t
    return _t


def dt(name):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[name]


def no_error():
    assert native.q8_device_error() == 0


def host(cache):
    return [x.cpu().numpy() for x in cache]


def dev(x, dtype=None):
    x = torch().from_numpy(np.ascontiguousarray(x)).to("cuda")
    return x if dtype is None else x.to(dtype)


def i32(x):
    return torch().tensor(x, dtype=torch().int32, device="cuda")


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and a.tobytes() == b.tobytes()


def filled(kind, rows, n_pos, kv_heads, dim, seed, lead=0):
    """A cache of random values, `lead` above zero, as planes on the host and on the device."""
    r = np.random.default_rng(seed)
    planes = []
    for _ in range(2):
        x = r.standard_normal((rows, kv_heads, n_pos, dim), dtype=np.float32) + np.float32(lead)
        codes, words = kr.quantise(x, kind)
        planes += [kr.pack(codes, kind), words]
    return planes, tuple(dev(p) for p in planes)


# ------------------------------------------------------------ store and load

def stored(planes, x, at, pos, lens, kind, n_pos):
    """planes[at], planes[at + 1] with x [rows][T][kv_heads][D] stored."""
    codes, words = kr.quantise(x, kind)
    codes = kr.pack(codes, kind)
    for m in range(x.shape[0]):
        for t in range(x.shape[1] if lens is None else min(x.shape[1], max(0, lens[m]))):
            if 0 <= pos[m] + t < n_pos:
                planes[at][m, :, pos[m] + t] = codes[m, t]
                planes[at + 1][m, :, pos[m] + t] = words[m, t]


def store_and_check(kind, src, rows, T, kv_heads, dim, n_pos, pos, lens=None, seed=0, error=0, x=None, pad=0):
    t = torch()
    r = np.random.default_rng(seed)
    width = kv_heads * dim
    qkv = r.standard_normal((rows, T, 6 * width + pad), dtype=np.float32) * 2 if x is None else x
    qkv = dev(qkv, dt(src))
    k, v = qkv[..., 4 * width:5 * width], qkv[..., 5 * width:6 * width]
    want, cache = filled(kind, rows, n_pos, kv_heads, dim, seed + 1)
    for at, f in ((0, k), (2, v)):
        stored(want, f.float().cpu().numpy().reshape(rows, T, kv_heads, dim), at, pos, lens, kind, n_pos)
    native.kvq_store(k, v, i32(pos), cache, lens=None if lens is None else i32(lens))
    got = host(cache)
    assert native.q8_device_error() == error
    for a, b in zip(got, want):
        if a.dtype == np.uint8 or a.dtype == np.int8:
            assert np.array_equal(a, b)
        else:                                    # (a zero's sign, a NaN's bits)
            assert np.array_equal(a, b, equal_nan=True)
    # read back
    for dst in FLOATS:
        both = t.full((rows, T, 2 * width + 8), 7.0, device="cuda", dtype=dt(dst))
        ko, vo = both[..., :width], both[..., width + 8:]
        native.kvq_load(cache, ko, vo, pos=i32(pos), lens=None if lens is None else i32(lens))
        for at, out in ((0, ko), (2, vo)):
            with np.errstate(over="ignore"):      # (the largest values round up)
                f = kr.values(want[at], want[at + 1], kind).astype(np.float32)
            exp = t.full((rows, T, width), 7.0, dtype=dt(dst))
            for m in range(rows):
                for i in range(T if lens is None else min(T, max(0, lens[m]))):
                    if 0 <= pos[m] + i < n_pos:
                        exp[m, i] = t.from_numpy(f[m, :, pos[m] + i].reshape(-1)).to(dt(dst))
            assert t.equal(t.nan_to_num(out.cpu().float(), 9e9), t.nan_to_num(exp.float(), 9e9))
        assert (both[..., width:width + 8] == 7).all()
        assert native.q8_device_error() == error


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src", FLOATS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_store_dims(kind, src, dim):
    store_and_check(kind, src, 3, 5, 2, dim, 40, [0, 35, 17], seed=dim)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,T,kv_heads", [(1, 1, 1), (1, 1, 8), (64, 1, 8), (256, 1, 2), (1, 2, 5), (2, 7, 3),
                                             (1, 15, 4), (1, 16, 4), (3, 17, 1), (1, 31, 2), (1, 33, 2), (2, 129, 1)])
def test_store_sizes(kind, rows, T, kv_heads):
    pos = [(5 * m) % 11 for m in range(rows)]
    store_and_check(kind, "f32", rows, T, kv_heads, 128, T + 11, pos, seed=rows + T)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,T,kv_heads,dim", [(1, 4001, 9, 160), (2, 9001, 5, 64), (3, 7000, 8, 128)])
def test_store_long_prompts(kind, rows, T, kv_heads, dim):
    """Several tokens a thread, in turns."""
    store_and_check(kind, "bf16", rows, T, kv_heads, dim, T + 5, list(range(rows)), lens=[T, T - 700, 3][:rows], seed=T)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("rows,T,kv_heads,dim", [(1, 401, 8, 128), (1, 701, 8, 128), (1, 2051, 8, 128), (3, 1003, 5, 96)])
def test_store_prompts_between_short_and_long(kind, src, rows, T, kv_heads, dim):
    """Several tokens a thread: stores in one turn, loads in one and two (on 148 to 160 SMs; four in f32), none of
    whose shares T is a multiple of."""
    lens = [T - 13, T, 517][:rows]
    store_and_check(kind, src, rows, T, kv_heads, dim, T + 3, [2, 0, 3][:rows], lens=lens, seed=T)
    store_and_check(kind, src, rows, T, kv_heads, dim, T - 5, [0, -3, 2][:rows], seed=T + 1, error=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src", FLOATS)
def test_long_prompts_are_their_pieces(kind, src):
    """The longest walks of a store and a load against calls of some tokens each."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(12)
    qkv = t.randn(2, 17001, 6 * 1024, device="cuda", generator=g).to(dt(src))
    k, v = qkv[..., 4096:5120], qkv[..., 5120:]
    whole, pieces = (native.kvq_cache(kind, 2, 17010, 8, 128) for _ in range(2))
    pos, lens = [3, 0], [17001, 16400]
    native.kvq_store(k, v, i32(pos), whole, lens=i32(lens))
    for a in range(0, 17001, 97):
        native.kvq_store(k[:, a:a + 97], v[:, a:a + 97], i32([p + a for p in pos]), pieces, lens=i32([n - a for n in lens]))
    for x, y in zip(whole, pieces):
        assert t.equal(x.view(t.uint8), y.view(t.uint8))
    outs = [t.zeros(2, 17001, 2048, device="cuda", dtype=dt(src)) for _ in range(2)]
    native.kvq_load(whole, outs[0][..., :1024], outs[0][..., 1024:], pos=i32(pos), lens=i32(lens))
    for a in range(0, 17001, 97):
        part = outs[1][:, a:a + 97]
        native.kvq_load(whole, part[..., :1024], part[..., 1024:], pos=i32([p + a for p in pos]), lens=i32([n - a for n in lens]))
    assert t.equal(*outs)
    no_error()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src", FLOATS)
def test_store_padded_batches(kind, src):
    store_and_check(kind, src, 6, 70, 2, 64, 90, [0, 1, 20, 5, 7, 3], lens=[70, 0, 1, -3, 1 << 30, 33], seed=5, pad=64)


@pytest.mark.parametrize("kind", KINDS)
def test_store_outside_the_cache(kind):
    """Such tokens are not stored and set the device error; the others are."""
    store_and_check(kind, "f32", 4, 9, 2, 64, 20, [15, -4, 0, 20], seed=6, error=2)
    store_and_check(kind, "f32", 3, 9, 2, 64, 20, [15, -4, 20], lens=[5, 0, 0], seed=6)
    store_and_check(kind, "f32", 2, 3, 2, 64, 20, [2 ** 31 - 1, -2 ** 31], seed=6, error=2)


@pytest.mark.parametrize("kind", KINDS)
def test_store_of_odd_values(kind):
    x = np.random.default_rng(8).standard_normal((1, 24, 6 * 64), dtype=np.float32)
    x[0, 0] = 0
    x[0, 1] = -0.0
    x[0, 2] = 5.25
    x[0, 3] = -5.25
    x[0, 4] *= 1e-42                              # subnormal
    x[0, 5] *= 1e-38
    x[0, 6] *= 1e38
    x[0, 7] *= 60000
    x[0, 8] = np.tile([0.5, 127.0, -3.5, 2.5], 96)   # halves of an i8 step of 1
    x[0, 9] = np.tile([0.0, 15.0, 7.5, 0.5], 96)     # of a u4 step of 1
    x[0, 10] *= 1e-8                              # below binary16
    x[0, 11] += 1000
    x[0, 12, 300] = np.nan
    x[0, 13, 260] = np.inf
    x[0, 14, 383] = -np.inf
    x[0, 15] = np.finfo(np.float32).max * np.where(np.arange(384) % 2, 1, -1)
    x[0, 16] = 65504
    x[0, 17] = 65519.996
    x[0, 18] = 65520
    x[0, 19] = np.where(np.arange(384) % 32 == 0, -65504, 65504)
    x[0, 20] = np.where(np.arange(384) % 32 == 0, -2.0 ** -24, 0)
    x[0, 21] = np.finfo(np.float32).tiny
    x[0, 22] = np.where(np.arange(384) % 32 == 7, 1e4, 1e-4)
    store_and_check(kind, "f32", 1, 24, 1, 64, 24, [0], x=x)


@pytest.mark.parametrize("kind", KINDS)
def test_store_rounds_as_the_format_says_near_halves(kind):
    """Quotients within a few steps of a half, where a reciprocal in place of the division would differ."""
    r = np.random.default_rng(9)
    x = np.zeros((1, 400, 6, 32), dtype=np.float32)
    top = (1 + r.random((400, 6, 1))).astype(np.float32)
    half = r.integers(0, 14 if kind == "u4" else 126, (400, 6, 32)) + 0.5
    step = top / np.float32(15 if kind == "u4" else 127)
    if kind == "u4":
        step = step.astype(np.float16).astype(np.float32)
    x[0] = (half * step).astype(np.float32)
    x[0] = np.nextafter(x[0], np.where(r.random(x[0].shape) < 0.5, np.float32(9), np.float32(0)))
    x[0, :, :, 0], x[0, :, :, 1] = 0, top[..., 0]
    store_and_check(kind, "f32", 1, 400, 1, 32, 400, [0], x=x.reshape(1, 400, 192))


@pytest.mark.parametrize("kind", KINDS)
def test_store_rounds_next_to_exact_halves(kind):
    """Steps that are powers of two: every half of them, and its neighbours on both sides."""
    most = 15 if kind == "u4" else 127
    half = (np.arange(most, dtype=np.float32) + np.float32(0.5))
    near = np.concatenate([half, np.nextafter(half, np.float32(0)), np.nextafter(half, np.float32(999))])
    near = np.concatenate([near, np.nextafter(near, np.float32(0)), -near if kind == "i8" else near])
    n = (len(near) + 29) // 30
    x = np.zeros((1, 12 * n, 6, 32), dtype=np.float32)
    for i, k in enumerate((-20, -10, -3, -1, 0, 1, 2, 5, 9, 11, -14, 3)):
        for b in range(n):
            part = near[30 * b:30 * b + 30]
            x[0, i * n + b, :, :len(part)] = part * np.float32(2.0 ** k)
            x[0, i * n + b, :, 31] = most * np.float32(2.0 ** k)          # (and the least, 0, at 30)
    store_and_check(kind, "f32", 1, 12 * n, 1, 32, 12 * n, [0], x=x.reshape(1, 12 * n, 192))
    want = kr.quantise(x[0, 5 * n:6 * n, 0], kind)[0]
    assert want.max() == most and len(np.unique(want)) > most


@pytest.mark.parametrize("kind", KINDS)
def test_store_strides(kind):
    """Tokens before rows, rows of separate tensors, one row's columns."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(3)
    big = t.randn(9, 4, 2, 96, device="cuda", generator=g)          # [T][rows][K and V][width]
    k, v = big[:, :, 0].transpose(0, 1), big[:, :, 1].transpose(0, 1)
    want, cache = filled(kind, 4, 12, 1, 96, 0)
    pos = [0, 3, 1, 2]
    for at, f in ((0, k), (2, v)):
        stored(want, f.cpu().numpy().reshape(4, 9, 1, 96), at, pos, None, kind, 12)
    native.kvq_store(k, v, i32(pos), cache)
    for a, b in zip(host(cache), want):
        assert same_bits(a, b)
    out = t.zeros_like(big)
    native.kvq_load(cache, out[:, :, 0].transpose(0, 1), out[:, :, 1].transpose(0, 1), pos=i32(pos))
    exp = kr.values(want[0], want[1], kind).astype(np.float32)
    for m in range(4):
        assert np.array_equal(out[:, m, 0].cpu().numpy(), exp[m, 0, pos[m]:pos[m] + 9])
    no_error()
    for bad in (k[..., :64], k[:, :, ::2], k.double(), k.cpu(), k[:3]):
        with pytest.raises((ValueError, TypeError, native.Q8Error)):
            native.kvq_store(bad, v, i32(pos), cache)
    with pytest.raises(ValueError):
        native.kvq_store(k, v.contiguous(), i32(pos), cache)
    with pytest.raises(native.Q8Error):
        native.kvq_load(cache, out[:, :1, 0].expand(9, 4, 96).transpose(0, 1), out[:, :1, 1].expand(9, 4, 96).transpose(0, 1))


@pytest.mark.parametrize("kind", KINDS)
def test_load_defaults_and_the_whole_cache(kind):
    planes, cache = filled(kind, 2, 300, 3, 64, 4, lead=0.5)
    t = torch()
    k, v = t.empty(2, 300, 192, device="cuda"), t.empty(2, 300, 192, device="cuda")
    native.kvq_load(cache, k, v)
    for got, at in ((k, 0), (v, 2)):
        exp = kr.entry_major(kr.values(planes[at], planes[at + 1], kind)).astype(np.float32)
        assert np.array_equal(got.cpu().numpy(), exp)
    no_error()


# ------------------------------------------------------------- attention

class Attn:
    """One call's inputs, seeded; q and out are columns of wider rows."""

    def __init__(self, kind, pos, heads, kv_heads, dim, n_pos, window=-1, sinks=0, acc=True, seed=0, pad=0, lead=0.3):
        t = torch()
        r = np.random.default_rng(seed)
        rows = len(pos)
        self.kind, self.heads, self.kv_heads, self.dim, self.n_pos = kind, heads, kv_heads, dim, n_pos
        self.window, self.sinks, self.pos = window, sinks, list(pos)
        self.planes, self.cache = filled(kind, rows, n_pos, kv_heads, dim, seed + 1, lead)
        self.wide = dev(r.standard_normal((rows, heads * dim + pad), dtype=np.float32))
        self.q = self.wide[:, :heads * dim]
        self.posd = i32(self.pos)
        self.acc = dev(r.random((rows, kv_heads, n_pos), dtype=np.float32)) if acc else None
        self.wide_out = t.full((rows, heads * dim + pad), 7.0, device="cuda")
        self.out = self.wide_out[:, :heads * dim]
        self.ws = native.kvq_attn_workspace(rows, heads, kv_heads, dim, n_pos, window, sinks, acc)

    def call(self, stream=None, scale=None):
        native.kvq_attn_decode(self.q, self.cache, self.posd, self.out, self.ws, self.heads, window=self.window,
                               sinks=self.sinks, acc=self.acc, stream=stream, scale=scale)

    def want(self, scale=None):
        f = lambda x: x.cpu().double().numpy()  # noqa: E731
        p = self.planes
        vals = [kr.values(p[i], p[i + 1], self.kind, spread) for spread in (False, True) for i in (0, 2)]
        return kr.attn(f(self.q), *vals, self.pos, self.heads, self.window, self.sinks,
                       self.dim ** -0.5 if scale is None else scale, None if self.acc is None else f(self.acc))

    def push(self):
        """The host's planes to the device."""
        for d, p in zip(self.cache, self.planes):
            d.copy_(dev(p))

    def compare(self, want):
        got = self.out.cpu().double().numpy()
        assert np.all(np.abs(got - want[0]) <= want[1]), float(np.max(np.abs(got - want[0]) / np.maximum(want[1], 1e-300)))
        if self.acc is not None:
            a = self.acc.cpu().double().numpy()
            assert np.all(np.abs(a - want[2]) <= want[3]), float(np.max(np.abs(a - want[2]) - want[3]))
        no_error()

    def check(self, scale=None):
        want = self.want(scale)
        self.call(scale=scale)
        self.compare(want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("group", [2, 8])
def test_attn_dims(kind, dim, group):
    Attn(kind, [299, 0, 17], 2 * group, 2, dim, 300, seed=dim).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 9, 16, 21])
def test_attn_groups(kind, group):
    Attn(kind, [130, 64], 2 * group, 2, 64, 131, window=100, sinks=3, seed=group).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 1000, 1025])
def test_attn_lengths(kind, group, n):
    Attn(kind, [n - 1], group, 1, 128, n, seed=n).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 1, 2, 15, 64, 100, 199, 200, 201, 1 << 40])
@pytest.mark.parametrize("sinks", [0, 1, 4, 70, 200, 1 << 40])
def test_attn_window_and_sinks(kind, window, sinks):
    Attn(kind, [199, 99, 64, 0, 3], 4, 2, 32, 200, window=window, sinks=sinks, seed=window % 97 + sinks % 89).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1024, 4, 32), (128, 1, 64), (1024, 1024, 32), (71, 71, 128)])
def test_attn_many_heads(kind, heads, kv_heads, dim):
    Attn(kind, [90, 12], heads, kv_heads, dim, 91, window=60, sinks=1, seed=heads).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 3, 40, 256])
def test_attn_ragged_batches(kind, rows):
    pos = [(37 * i * i + 11) % 400 - 1 for i in range(rows)]
    Attn(kind, pos, 8, 2, 64, 400, window=150, sinks=5, seed=rows, pad=5).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [4, 8])
def test_attn_one_long_row_and_short_ones(kind, heads):
    Attn(kind, [20000, 5, -1, 900], heads, 1, 64, 20001, seed=heads).check()
    Attn(kind, [30000], heads, 1, 96, 30001, seed=heads, acc=False).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attn_rows_without_entries(kind):
    """Zeros, acc as it was; columns behind the heads keep what they held."""
    a = Attn(kind, [-1, 40, -1], 8, 2, 64, 64, pad=8)
    a.check()
    assert (a.out[0] == 0).all() and (a.out[2] == 0).all() and (a.wide_out[:, a.heads * a.dim:] == 7).all()
    a = Attn(kind, [50, 3], 8, 2, 64, 64, window=0, sinks=0)
    old = a.acc.clone()
    a.call()
    assert (a.out == 0).all() and torch().equal(a.acc, old)


@pytest.mark.parametrize("kind", KINDS)
def test_attn_positions_outside_the_cache(kind):
    a = Attn(kind, [63, 64, -2, 5], 8, 2, 64, 64)
    a.pos = [63, -1, -1, 5]
    want = a.want()
    a.call()
    assert native.q8_device_error() == 2
    a.compare(want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [4, 8])
def test_attn_what_is_not_visible_does_not_matter(kind, heads):
    """NaN and the largest codes and words in entries behind the last one and outside the window."""
    a = Attn(kind, [150, 99, 20], heads, 1, 128, 256, window=50, sinks=3)
    want = a.want()
    for i, p in enumerate(a.planes):
        bad = p.copy()
        for m, pos in enumerate(a.pos):
            gone = [j for j in range(256) if j > pos or 3 <= j <= pos - 50]
            bad[m, :, gone] = np.nan if i % 2 else (255 if kind == "u4" else -128)
        a.planes[i] = bad
    a.push()
    a.call()
    a.compare(want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [8, 16])
@pytest.mark.parametrize("dim", [64, 96, 256])
def test_attn_blocks_of_nan_that_are_seen(kind, heads, dim):
    """A block of K reaches its head's whole output, a block of V its own values, nothing else."""
    a = Attn(kind, [499, 499, 30], heads, 2, dim, 500, seed=3)
    clean = a.want()
    a.planes[1][0, 0, 450, 1] = np.nan                    # K of K/V head 0, row 0
    a.planes[3][1, 1, 77, 0] = np.nan                     # V of head 1, row 1
    a.push()
    a.call()
    got, acc = a.out.cpu().double().numpy(), a.acc.cpu().double().numpy()
    half = heads // 2 * dim
    assert np.isnan(got[0, :half]).all() and np.isnan(acc[0, 0]).all()
    hit = np.zeros(clean[0].shape, dtype=bool)
    hit[0, :half] = True
    hit[1, half:] = np.arange(half) % dim < 32
    assert np.isnan(got[hit]).all() and np.all(np.abs(got - clean[0])[~hit] <= clean[1][~hit])
    ok = np.ones(acc.shape, dtype=bool)
    ok[0, 0] = False
    assert np.all(np.abs(acc - clean[2])[ok] <= clean[3][ok])
    no_error()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attn_queries_that_are_not_finite(kind, bad):
    """Their head is NaN, the others are not."""
    a = Attn(kind, [80, 40], 16, 2, 64, 100, acc=False)
    want = a.want()
    a.q[0, 5 * 64 + 9] = bad
    a.call()
    got = a.out.cpu().double().numpy()
    hit = np.zeros(got.shape, dtype=bool)
    hit[0, 5 * 64:6 * 64] = True
    assert np.isnan(got[hit]).all() and np.all(np.abs(got - want[0])[~hit] <= want[1][~hit])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [4, 8])
def test_attn_of_odd_magnitudes(kind, heads):
    for q_scale, k_scale, v_scale in ((1e-6, 1.0, 1.0), (1e-6, 3e4, 1.0), (30.0, 1.0, 1e4), (1e4, 1e-3, 1e-6),
                                      (1.0, 1e-4, 1.0), (0.0, 1.0, 1.0), (1e-30, 1.0, 1.0), (1e30, 1e-8, 1.0)):
        a = Attn(kind, [499, 40], heads, 1, 64, 500, seed=3, lead=0)
        a.wide.mul_(q_scale)
        a.q[:, :64] *= torch().logspace(-6, 0, 64, device="cuda")        # one head's values far apart
        for i, s in ((1, k_scale), (3, v_scale)):
            a.planes[i] = np.clip(a.planes[i].astype(np.float32) * np.float32(s), -6e4, 6e4).astype(a.planes[i].dtype)
        a.push()
        a.check()
    a = Attn(kind, [499, 40], heads, 1, 64, 500, seed=4)                 # masks of the type's lowest value
    a.q.abs_()
    low = 6e4 if kind == "u4" else 1e30
    a.planes[0][:, :, ::3] = 0 if kind == "u4" else -127
    a.planes[1][:, :, ::3] = [0, -low] if kind == "u4" else low / 127
    a.push()
    a.check()


@pytest.mark.parametrize("kind", KINDS)
def test_attn_scales(kind):
    for scale in (0.0, -0.5, 1.0, 1e-20):
        Attn(kind, [120, 7], 4, 1, 64, 121, seed=2).check(scale)


def planes_of(kind, k, v, n_pos):
    """Planes that stand for k and v [rows][n][D] exactly, of given (code, words) pairs a value array."""
    out = []
    for codes, words in (k, v):
        out += [kr.pack(codes[:, None], kind), words[:, None]]
    return out


def run_planes(kind, q, planes, scale, acc=True):
    """kvq_attn_decode of q [rows][heads][D] on one K/V head's planes: out, weights."""
    t = torch()
    rows, heads, dim = q.shape
    n = planes[0].shape[2]
    out = t.empty(rows, heads * dim, device="cuda")
    w = t.zeros(rows, 1, n, device="cuda") if acc else None
    native.kvq_attn_decode(dev(q.reshape(rows, -1), t.float32), tuple(dev(p) for p in planes), i32([n - 1] * rows), out,
                           native.kvq_attn_workspace(rows, heads, 1, dim, n, acc=acc), heads, scale=scale, acc=w)
    no_error()
    return out.double().cpu().numpy().reshape(rows, heads, dim), w.double().cpu().numpy()[:, 0] if acc else None


def in_range(got, want, tol):
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [2, 4, 5, 8])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("n,at", [(16, 0), (300, 5)])
def test_small_weights_beside_large_ones_of_no_value(kind, heads, dim, n, at):
    """All of the weight but 2^-4 to 2^-95 of it stands on entries of no value."""
    q, k, v = ap.small_weights(heads, dim, n, at)
    rows, r = k.shape[0], np.random.default_rng(dim)
    nb = dim // 32
    big = np.zeros((rows, n), dtype=bool)
    big[:, at::16] = True
    if kind == "i8":
        kc = np.zeros((rows, n, dim), np.int8)
        kc[:, :, 0] = np.where(big, 1, -3)
        kw = np.where(big, k[:, :, 0], 0.125)[..., None].repeat(nb, 2).astype(np.float32)
        vc = np.where(big[..., None], 0, r.integers(64, 128, (rows, n, dim))).astype(np.int8)
        vw = np.full((rows, n, nb), 1 / 64, np.float32)
    else:
        kc = np.zeros((rows, n, dim), np.uint8)
        kw = np.stack((np.zeros_like(k[:, :, :nb]), k[:, :, :1].repeat(nb, 2)), -1).astype(np.float16)
        vc = np.where(big[..., None], 0, r.integers(0, 16, (rows, n, dim))).astype(np.uint8)
        vw = np.stack((np.full((rows, n, nb), 1 / 16), np.where(big[..., None], 0, 1).repeat(nb, 2)), -1).astype(np.float16)
    planes = planes_of(kind, (kc, kw), (vc, vw), n)
    k, v = (kr.values(planes[i], planes[i + 1], kind)[:, 0] for i in (0, 2))
    want, p = ap.exact(q, k, v)
    got, acc = run_planes(kind, q, planes, ap.SCALE)
    in_range(got, want, ap.small_weights_bound(want, n))
    in_range(acc, p.sum(1), ap.small_weights_bound(p.sum(1), n) + (heads + 1) * ap.U * p.sum(1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [64, 600])
def test_weights_that_cancel(kind, heads, dim, n):
    q, k, v = ap.cancelling_weights(heads, dim, n)
    want, _ = ap.exact(q, k, v)
    nb = dim // 32
    if kind == "i8":
        parts = [(x.astype(np.int8), np.ones((1, n, nb), np.float32)) for x in (k, v)]
    else:     # m = -1, s = 1 or 2: codes 1 and 0
        parts = [((x > -1).astype(np.uint8), np.tile(np.array([s, -1], np.float16), (1, n, nb, 1))) for x, s in ((k, 1), (v, 2))]
    planes = planes_of(kind, *parts, n)
    assert np.array_equal(kr.values(planes[0], planes[1], kind)[:, 0], k)
    assert np.array_equal(kr.values(planes[2], planes[3], kind)[:, 0], v)
    # u4: the score is a difference of sums of q, 2^-10 at most (8u).  V is m + s code (at most 1 + 2) or
    # m + 15 s less s (15 - code) (29 and at most 30): sums of weights times 30.  The first ones': one
    # rounding a term, of 16 kinds of entries (by their place of 16) N = ceil(n / 16) terms each, so
    # u 30 N (N + 1) / 2 a kind, 16 kinds over n weights: 30 u (N + 1) / 2.  The products': chains of 32
    # entries, 16 of them negative, six additions truncated by 2u of at most 16 * 30, over 32 weights: 180u;
    # the chains' sums, rounded, n / 32 of them, u 16 * 30 each, over n: 15u.
    more = (8 + 15 * (n // 16 + 2) + 180 + 15) * ap.U if kind == "u4" else 0
    in_range(run_planes(kind, q, planes, ap.SCALE)[0], want, ap.cancelling_weights_bound(want, n) + more)


@pytest.mark.parametrize("heads", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [64, 600])
def test_weights_that_cancel_in_blocks_that_span_their_codes(heads, dim, n):
    """As above in u4, with V of +-15/16 as codes 15 and 0 (what kvq_store makes of such a block)."""
    q, k, v = ap.cancelling_weights(heads, dim, n)
    v[:, :, 1::2] *= -1                              # (both codes in a block)
    nb = dim // 32
    kp = ((k > -1).astype(np.uint8), np.tile(np.array([1, -1], np.float16), (1, n, nb, 1)))
    vp = ((v > 0).astype(np.uint8) * 15, np.tile(np.array([0.125, -0.9375], np.float16), (1, n, nb, 1)))
    planes = planes_of("u4", kp, vp, n)
    assert np.array_equal(kr.values(planes[2], planes[3], "u4")[:, 0], v * 0.9375)
    want, _ = ap.exact(q, k, v * 0.9375)
    # the score 8u as above; the terms are at most 15/16 and 15/8: additions of at most 16 entries' 15/8 in
    # a chain, truncated six times by 2u, over 32 weights (12u), of 16 kinds of entries 15/16 (N + 1) / 2 u
    in_range(run_planes("u4", q, planes, ap.SCALE)[0], want,
             ap.cancelling_weights_bound(want, n) + (8 + 12 + (n // 16 + 2) / 2) * ap.U)


@pytest.mark.parametrize("heads", [4, 7, 8])
@pytest.mark.parametrize("dim", [64, 96, 256])
def test_low_parts_of_q(heads, dim):
    """Scores that are the difference of two keys' products, whose leading 16 bits cancel (i8: codes of 1 and -1)."""
    q, k, v = ap.low_parts_of_q("f16", heads, dim)
    want, p = ap.exact(q, k, v)
    nb, n = dim // 32, k.shape[1]
    planes = planes_of("i8", ((k / 2.0 ** 15).astype(np.int8), np.full((1, n, nb), 2.0 ** 15, np.float32)),
                       (v.astype(np.int8), np.ones((1, n, nb), np.float32)), n)
    tol = ap.low_parts_of_q_bound(want, "f16", 8, dim)
    in_range(run_planes("i8", q, planes, ap.SCALE)[0], want, tol)


@pytest.mark.parametrize("kind,heads,dim,n", [
    ("i8", 8, 256, 9000), ("i8", 5, 32, 30000), ("i8", 1, 64, 60000), ("u4", 8, 128, 30000), ("u4", 3, 32, 60000),
    ("u4", 1, 256, 40000), ("u4", 7, 96, 20000), ("i8", 4, 160, 20000)])
def test_every_part_of_a_long_row_counts(kind, heads, dim, n):
    """V is 1 in one slice of the row a column, so that a part lost or misweighed in the join moves a column."""
    r = np.random.default_rng(n + dim)
    q = r.standard_normal((1, heads, dim)).astype(np.float32).astype(np.float64)
    nb = dim // 32
    kc, kw = kr.quantise(r.standard_normal((1, n, dim)).astype(np.float32), kind)
    vc = ap.sliced_values(n, dim)[None]
    vw = np.ones((1, n, nb), np.float32) if kind == "i8" else np.tile(np.array([1, 0], np.float16), (1, n, nb, 1))
    planes = planes_of(kind, (kc, kw), (vc.astype(kc.dtype), vw), n)
    k, spread = (kr.values(planes[0], planes[1], kind, s)[0, 0] for s in (False, True))
    scale = dim ** -0.5
    want, p = ap.exact(q * scale / np.log(2), k[None], vc)
    got, acc = run_planes(kind, q, planes, scale)
    # (a score's bound by what a value is made of, twice: sums may be truncated)
    tol = 2 * ap.long_row_bound(q[0], spread, want[0], scale)
    in_range(got[0], want[0], tol)
    in_range(acc[0], p[0].sum(0), 2 * ap.long_row_bound(q[0], spread, p[0], scale).sum(0) + (heads + 1) * ap.U * p[0].sum(0))


@pytest.mark.parametrize("kind", KINDS)
def test_attn_repeats_bit_for_bit_on_two_streams(kind):
    t = torch()
    a = [Attn(kind, [3000, 100 + i, 7], 8, 2, 128, 3001, seed=i, acc=False) for i in range(2)]
    want = []
    for x in a:
        x.call()
        want.append(x.out.clone())
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in a]
    for _ in range(20):
        for x, s in zip(a, streams):
            x.call(stream=s)
        t.cuda.synchronize()
        for x, w in zip(a, want):
            assert t.equal(x.out, w)
    no_error()


@pytest.mark.parametrize("kind", KINDS)
def test_attn_beyond_32_bits(kind):
    """Entries whose bytes lie more than 2^32 into their plane."""
    t = torch()
    dim, n_pos = 256, (1 << 25) + 4096 if kind == "u4" else (1 << 24) + 4096
    cache = native.kvq_cache(kind, 1, n_pos, 1, dim)
    planes, part = filled(kind, 1, 600, 1, dim, 5)
    for c, p in zip(cache, part):
        c[:, :, n_pos - 600:] = p
    q = t.randn(1, 4 * dim, device="cuda", generator=t.Generator(device="cuda").manual_seed(1))
    out = t.zeros(1, 4 * dim, device="cuda")
    native.kvq_attn_decode(q, cache, i32([n_pos - 1]), out, native.kvq_attn_workspace(1, 4, 1, dim, n_pos, 600), 4, window=600)
    vals = [kr.values(planes[i], planes[i + 1], kind, s) for s in (False, True) for i in (0, 2)]
    want, tol, _, _ = kr.attn(q.cpu().double().numpy(), *vals, [599], 4, -1, 0, dim ** -0.5)
    in_range(out.cpu().double().numpy(), want, tol)
    # the same entries stored and read back there
    k = t.randn(1, 300, dim, device="cuda", generator=t.Generator(device="cuda").manual_seed(2))
    ko, vo = t.empty_like(k), t.empty_like(k)
    native.kvq_store(k, k, i32([n_pos - 300]), cache)
    native.kvq_load(cache, ko, vo, pos=i32([n_pos - 300]))
    codes, words = kr.quantise(k.cpu().numpy(), kind)
    exp = kr.values(kr.pack(codes, kind), words, kind).astype(np.float32)
    assert np.array_equal(ko.cpu().numpy(), exp) and np.array_equal(vo.cpu().numpy(), exp)
    # and moved
    acc = t.zeros(1, 1, n_pos, device="cuda")
    acc[..., n_pos - 300:] = 1
    ws = t.zeros(native.kvq_evict_workspace(1, 1, 300), dtype=t.uint8, device="cuda")
    native.kvq_evict(cache, i32([n_pos - 1]), acc, i32([0]), acc, ws, 300)
    native.kvq_load(cache, ko, vo)
    assert np.array_equal(ko.cpu().numpy(), exp) and np.array_equal(vo.cpu().numpy(), exp)
    no_error()


# ------------------------------------------------------------- eviction

def evict_and_check(kind, pos, kv_heads, dim, n_pos, budget, sinks, recent, seed=0, in_place=False, kept=True, acc=None):
    t = torch()
    rows = len(pos)
    planes, cache = filled(kind, rows, n_pos, kv_heads, dim, seed)
    r = np.random.default_rng(seed + 9)
    if acc is None:
        acc = (np.maximum(r.standard_normal((rows, kv_heads, n_pos)), 0) ** 3).astype(np.float32)
    fine = [p if -1 <= p < n_pos else -1 for p in pos]
    want, new_pos, new_acc, want_kept = kr.evict(planes, fine, acc, budget, sinks, recent)
    for m, p in enumerate(pos):
        if p != fine[m]:
            new_pos[m] = p
    posd, accd = i32(pos), dev(acc)
    npos, nacc = (posd, accd) if in_place else (t.full_like(posd, 77), t.full_like(accd, 77))
    keptd = t.full((rows, kv_heads, budget), 77, dtype=t.int32, device="cuda") if kept else None
    ws = t.full((native.kvq_evict_workspace(rows, kv_heads, budget),), 7, dtype=t.uint8, device="cuda")
    native.kvq_evict(cache, posd, accd, npos, nacc, ws, budget, sinks=sinks, recent=recent, kept=keptd)
    for a, b in zip(host(cache), want):
        assert same_bits(a, b)
    assert np.array_equal(npos.cpu().numpy(), new_pos) and np.array_equal(nacc.cpu().numpy(), new_acc, equal_nan=True)
    if kept:
        assert np.array_equal(keptd.cpu().numpy(), want_kept)
    assert native.q8_device_error() == (2 if list(pos) != fine else 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_evict_dims(kind, dim):
    evict_and_check(kind, [299, 150, 149, -1, 20], 2, dim, 300, 150, 3, 40, seed=dim)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,budget", [(2, 1), (3, 2), (33, 32), (257, 64), (600, 599), (2100, 1000), (5000, 3000), (9000, 8999)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_sizes(kind, n, budget, in_place):
    evict_and_check(kind, [n - 1, n // 2], 3, 64, n, budget, min(1, budget - 1), budget // 3, seed=n, in_place=in_place)


@pytest.mark.parametrize("kind", KINDS)
def test_evict_batches_ties_and_bad_positions(kind):
    evict_and_check(kind, [(i * 7) % 200 for i in range(256)], 2, 32, 200, 90, 4, 10, kept=False)
    evict_and_check(kind, [199, 200, -2, 30], 2, 128, 200, 90, 4, 10)
    acc = np.random.default_rng(1).integers(0, 3, (2, 2, 400)).astype(np.float32)
    acc[0, 0, ::5] = np.nan
    evict_and_check(kind, [399, 350], 2, 96, 400, 111, 2, 3, acc=acc)
    evict_and_check(kind, [399, 350], 2, 64, 400, 50, 20, 30, acc=acc)


@pytest.mark.parametrize("kind", KINDS)
def test_evict_long_rows(kind):
    evict_and_check(kind, [39999, 30000], 2, 128, 40000, 25000, 16, 500, seed=3)
    evict_and_check(kind, [69999], 1, 64, 70000, 40000, 4, 100, seed=4, in_place=True)


# ------------------------------------------------------- a run of them

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("graph", [False, True])
def test_a_prompt_and_decode_steps_together(kind, graph):
    """A padded batch of prompts stored, then steps of store, attention with weights and, half way,
    eviction, on one workspace (also replayed from a graph), against the plain forms in turn."""
    t = torch()
    rows, heads, kv_heads, dim, n_pos, budget = 3, 8, 2, 64, 96, 40
    width, lens = kv_heads * dim, [50, 31, 47]
    r = np.random.default_rng(11)
    prompt = r.standard_normal((rows, 50, 2 * width), dtype=np.float32)
    steps = r.standard_normal((12, rows, 1, (heads + 2 * kv_heads) * dim), dtype=np.float32)
    cache = native.kvq_cache(kind, rows, n_pos, kv_heads, dim)
    zero, pos, acc = i32([0] * rows), i32([n - 1 for n in lens]), t.zeros(rows, kv_heads, n_pos, device="cuda")
    p = dev(prompt)
    native.kvq_store(p[..., :width], p[..., width:], zero, cache, lens=i32(lens))
    qkv, out = t.empty(rows, 1, (heads + 2 * kv_heads) * dim, device="cuda"), t.empty(rows, heads * dim, device="cuda")
    nbytes = max(native.kvq_attn_decode_workspace(rows, heads, kv_heads, dim, n_pos, acc=True),
                 native.kvq_evict_workspace(rows, kv_heads, budget))
    ws = t.zeros(nbytes, dtype=t.uint8, device="cuda")
    k, v = qkv[..., heads * dim:heads * dim + width], qkv[..., heads * dim + width:]

    def step():
        pos.add_(1)
        native.kvq_store(k, v, pos, cache)
        native.kvq_attn_decode(qkv[:, 0], cache, pos, out, ws, heads, acc=acc)

    def evict():
        native.kvq_evict(cache, pos, acc, pos, acc, ws, budget, sinks=2, recent=8)

    run = step
    if graph:
        keep = [x.clone() for x in cache + (pos, acc)]
        qkv.copy_(dev(steps[0]))
        s = t.cuda.Stream()
        s.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(s):
            step()
        t.cuda.current_stream().wait_stream(s)
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            step()
        for x, y in zip(cache + (pos, acc), keep):
            x.copy_(y)
        run = g.replay
    planes = [np.zeros_like(x) for x in host(cache)]
    for at, cols in ((0, slice(0, width)), (2, slice(width, None))):
        stored(planes, prompt[..., cols].reshape(rows, 50, kv_heads, dim), at, [0] * rows, lens, kind, n_pos)
    want_pos, want_acc, want_tol = [n - 1 for n in lens], np.zeros((rows, kv_heads, n_pos)), 0.0
    for i, x in enumerate(steps):
        qkv.copy_(dev(x))
        run()
        want_pos = [n + 1 for n in want_pos]
        for at, lo in ((0, heads * dim), (2, heads * dim + width)):
            stored(planes, x[..., lo:lo + width].reshape(rows, 1, kv_heads, dim), at, want_pos, None, kind, n_pos)
        vals = [kr.values(planes[j], planes[j + 1], kind, s) for s in (False, True) for j in (0, 2)]
        want, tol, want_acc, acc_tol = kr.attn(x[:, 0, :heads * dim].astype(np.float64), *vals, want_pos, heads, -1, 0,
                                               dim ** -0.5, want_acc)
        want_tol = want_tol + acc_tol
        in_range(out.cpu().double().numpy(), want, tol)
        in_range(acc.cpu().double().numpy(), want_acc, want_tol)
        for a, b in zip(host(cache), planes):
            assert np.array_equal(a, b)
        assert pos.tolist() == want_pos
        if i == 5:
            got_acc = acc.cpu().numpy()            # (its own roundings decide what stays)
            evict()
            planes, new_pos, new_acc, _ = kr.evict(planes, want_pos, got_acc, budget, 2, 8)
            want_pos, want_acc = [int(n) for n in new_pos], new_acc.astype(np.float64)
            want_tol = 0.0
            assert np.array_equal(acc.cpu().numpy(), new_acc)
    no_error()


@pytest.mark.parametrize("kind", KINDS)
def test_one_workspace_serves_every_call(kind):
    """Sizes, kinds and attn_decode in turn on one workspace, never cleared."""
    t = torch()
    calls = [Attn(k, [n - 1, n // 3], h, kvh, d, n, seed=n)
             for k, h, kvh, d, n in ((kind, 8, 1, 128, 3000), ("u4", 4, 2, 64, 77), ("i8", 32, 4, 96, 900), (kind, 1, 1, 32, 5000))]
    ws = t.zeros(max(x.ws.numel() for x in calls) + 4096, dtype=t.uint8, device="cuda")
    fk = t.randn(2, 900, 64, device="cuda")
    ws2 = native.attn_decode_workspace(2, 8, 1, 64, 900)
    ws = t.zeros(max(ws.numel(), ws2), dtype=t.uint8, device="cuda")
    for _ in range(2):
        for x in calls:
            x.ws = ws
            x.check()
            o = t.empty(2, 512, device="cuda")
            native.attn_decode(t.ones(2, 512, device="cuda"), fk, fk, i32([899, 5]), o, ws, 8, 1)
    no_error()


def test_calls_run_on_the_callers_stream():
    """Behind a long kernel of that stream, which fills what they read."""
    t = torch()
    s = t.cuda.Stream()
    cache = native.kvq_cache("u4", 1, 64, 1, 64)
    k = t.zeros(1, 64, 64, device="cuda")
    x = t.randn(1, 64, 64, device="cuda")
    zero, ko, vo = i32([0]), t.empty_like(k), t.empty_like(k)
    t.cuda.synchronize()
    with t.cuda.stream(s):
        t.cuda._sleep(20_000_000)
        k.copy_(x)
    native.kvq_store(k, k, zero, cache, stream=s)
    native.kvq_load(cache, ko, vo, stream=s)
    s.synchronize()
    codes, words = kr.quantise(x.cpu().numpy(), "u4")
    assert np.array_equal(ko.cpu().numpy(), kr.values(kr.pack(codes, "u4"), words, "u4").astype(np.float32))
    no_error()


def test_binding_refuses_what_does_not_fit():
    t = torch()
    cache = native.kvq_cache("u4", 2, 32, 2, 64)
    q, out, pos, ws = t.zeros(2, 512, device="cuda"), t.zeros(2, 512, device="cuda"), i32([3, 4]), t.zeros(1 << 22, dtype=t.uint8, device="cuda")
    call = lambda c=cache, q=q, out=out, pos=pos, **kw: native.kvq_attn_decode(q, c, pos, out, ws, 8, **kw)  # noqa: E731
    call()
    for bad in (dict(q=q[:1]), dict(q=q.half()), dict(q=q.T), dict(out=out[:, :500]), dict(pos=pos.long()), dict(pos=pos[:1]),
                dict(c=cache[:2] + native.kvq_cache("i8", 2, 32, 2, 64)[2:]), dict(c=(cache[0].float(),) + cache[1:]), dict(c=(cache[0][:, :1],) + cache[1:]),
                dict(c=(cache[0], cache[1].float()) + cache[2:]), dict(c=tuple(x[:, :, ::2] for x in cache)), dict(acc=out)):
        with pytest.raises((ValueError, TypeError, native.Q8Error)):
            call(**bad)
    no_error()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dst", FLOATS)
@pytest.mark.parametrize("rows,T,place", [(1, 1, "apart"), (1, 1, "turned"), (4, 1, "rows"), (3, 4, "halves"), (1, 4, "rows")])
def test_load_with_buffers_between(kind, dst, rows, T, place):
    """K and V in one line of memory with pos, lens and the cache between them, whatever order they have."""
    t = torch()
    kv_heads, dim, n_pos, width = 2, 96, 9, 192
    planes, _ = filled(kind, rows, n_pos, kv_heads, dim, seed=rows + T)
    elt = t.empty((), dtype=dt(dst)).element_size()
    pos, lens = [(3 * m + 2) % (n_pos - T + 1) for m in range(rows)], [T] * rows
    line = t.full((1 << 20,), 85, dtype=t.uint8, device="cuda")

    def at(begin, x):
        """x's copy at byte `begin` of the line."""
        y = line[begin:begin + x.numel() * x.element_size()].view(x.dtype).view(x.shape)
        y.copy_(x)
        return y

    # (the row pitch of "rows": from a row's K over 64 KB and its V on to the next)
    pitch = {"apart": 0, "turned": 0, "rows": 1 << 17, "halves": 2 * T * width * elt}[place]
    k0, v0 = (1 << 17, 0) if place == "turned" else (0, T * width * elt) if place == "halves" else (0, 1 << 16)
    tok = 2 * width if place == "rows" else width
    ko, vo = (line[b:].view(dt(dst)).as_strided((rows, T, width), (pitch // elt, tok, 1)) for b in (k0, v0))
    mid = (1 << 19) if place == "halves" else (1 << 14)
    cache = tuple(at(mid + 8192 * i, dev(p)) for i, p in enumerate(planes))
    pos_d, lens_d = at(mid + 40960, i32(pos)), at(mid + 40960 + 1024, i32(lens))
    want = line.clone()
    exp = kr.values(planes[0], planes[1], kind).astype(np.float32), kr.values(planes[2], planes[3], kind).astype(np.float32)
    for begin, f in zip((k0, v0), exp):
        w = want[begin:].view(dt(dst)).as_strided((rows, T, width), (pitch // elt, tok, 1))
        for m in range(rows):
            x = f[m, :, pos[m]:pos[m] + T].transpose(1, 0, 2).reshape(T, width)
            w[m].copy_(dev(x, dt(dst)))
    native.kvq_load(cache, ko, vo, pos=pos_d, lens=lens_d)
    assert t.equal(line, want)
    no_error()
    if T > 1:                                       # K's second token is V's first
        with pytest.raises(native.Q8Error):
            native.kvq_load(cache, ko[:, :T - 1], ko[:, 1:], pos=pos_d)
    with pytest.raises(native.Q8Error):
        native.kvq_load(cache, ko, ko, pos=pos_d)
