"""GPU tests of attn_decode, kv_evict and head_sample against 64-bit forms."""
import math

import numpy as np
import pytest

import decode_ref as ref
from q8_quantized_projection_gb300 import native

pytestmark = pytest.mark.gpu


def torch():
    import torch as _t
    return _t


def dt(kv):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[kv]


def no_error():
    assert native.q8_device_error() == 0


# ------------------------------------------------------------- attn_decode

class Attn:
    """One call's inputs, seeded; q and out are columns of wider rows."""

    def __init__(self, kv, pos, heads, kv_heads, dim, n_pos, window=-1, sinks=0, acc=True, spread=1.0,
                 seed=0, pad=0):
        t = torch()
        g = t.Generator(device="cuda").manual_seed(seed)
        rows = len(pos)
        self.heads, self.kv_heads, self.dim, self.n_pos = heads, kv_heads, dim, n_pos
        self.window, self.sinks, self.pos = window, sinks, list(pos)
        self.wide = t.randn(rows, heads * dim + pad, device="cuda", generator=g) * spread
        self.q = self.wide[:, :heads * dim]
        self.k = t.randn(rows, n_pos, kv_heads * dim, device="cuda", generator=g).to(dt(kv))
        self.v = t.randn(rows, n_pos, kv_heads * dim, device="cuda", generator=g).to(dt(kv))
        self.posd = t.tensor(pos, dtype=t.int32, device="cuda")
        self.acc = t.rand(rows, kv_heads, n_pos, device="cuda", generator=g) if acc else None
        self.wide_out = t.full((rows, heads * dim + pad), 7.0, device="cuda")
        self.out = self.wide_out[:, :heads * dim]
        self.ws = native.attn_workspace(rows, heads, kv_heads, dim, n_pos, window, sinks, acc)

    def call(self, stream=None, scale=None):
        native.attn_decode(self.q, self.k, self.v, self.posd, self.out, self.ws, self.heads, self.kv_heads,
                           window=self.window, sinks=self.sinks, acc=self.acc, stream=stream, scale=scale)

    def want(self, scale=None):
        f = lambda x: x.cpu().double().numpy()  # noqa: E731
        return ref.attn(f(self.q), f(self.k), f(self.v), self.pos, self.heads, self.kv_heads, self.window,
                        self.sinks, self.dim ** -0.5 if scale is None else scale,
                        None if self.acc is None else f(self.acc))

    def check(self, scale=None):
        want, tol, acc, acc_tol = self.want(scale)
        self.call(scale=scale)
        got = self.out.cpu().double().numpy()
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))
        if self.acc is not None:
            a = self.acc.cpu().double().numpy()
            assert np.all(np.abs(a - acc) <= acc_tol), float(np.max(np.abs(a - acc) - acc_tol))
        no_error()


@pytest.mark.parametrize("kv", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 40, 64, 80, 96, 128, 136, 192, 256])
def test_attn_dims(kv, dim):
    Attn(kv, [299, 0, 17], 4, 2, dim, 300, seed=dim).check()


@pytest.mark.parametrize("kv", ["f32", "bf16"])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 9, 16, 21])
def test_attn_groups(kv, group):
    Attn(kv, [130, 64], 2 * group, 2, 64, 131, window=100, sinks=3, seed=group).check()


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("group,dim", [(8, 256), (5, 192), (6, 128), (8, 16), (4, 256), (1, 256), (2, 32)])
def test_attn_group_and_dim(kv, group, dim):
    Attn(kv, [70, 255, 3], 2 * group, 2, dim, 256, window=61, sinks=2, seed=group * dim).check()


@pytest.mark.parametrize("kv", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 1000, 1025])
def test_attn_lengths(kv, n):
    Attn(kv, [n - 1], 4, 1, 128, n, seed=n).check()


@pytest.mark.parametrize("window", [0, 1, 2, 15, 64, 100, 199, 200, 201, 1 << 40])
@pytest.mark.parametrize("sinks", [0, 1, 4, 70, 200, 1 << 40])
def test_attn_window_and_sinks(window, sinks):
    Attn("f32", [199, 99, 64, 0, 3], 4, 2, 32, 200, window=window, sinks=sinks, seed=window % 97 + sinks % 89).check()


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 24, 64, 72, 88, 96, 104, 128])
@pytest.mark.parametrize("group,n", [(5, 17), (6, 1), (7, 64), (8, 300), (16, 65)])
def test_attn_eight_heads_of_16_bit_caches(kv, dim, group, n):
    """The products on the matrix instructions: heads padded to whole steps, entries to whole stages."""
    Attn(kv, [n - 1, n // 2, n // 3], 2 * group, 2, dim, n, window=70, sinks=2, seed=dim + n).check()


@pytest.mark.parametrize("kv", ["f16", "bf16"])
def test_attn_eight_heads_of_odd_magnitudes(kv):
    t = torch()
    for q_scale, k_scale in ((1e-6, 1.0), (1e-6, 3e4), (30.0, 1.0), (1e4, 1e-3), (1.0, 1e-4), (0.0, 1.0)):
        a = Attn(kv, [499, 40], 8, 1, 64, 500, seed=3)
        a.wide.mul_(q_scale)
        a.q[:, :64] *= t.logspace(-6, 0, 64, device="cuda")        # one head's values far apart
        a.k.copy_((a.k.float() * k_scale).clamp(-6e4, 6e4).to(a.k.dtype))     # (within f16)
        a.check()
    a = Attn(kv, [499, 40], 8, 1, 64, 500, seed=4)                 # masks of the type's lowest value
    a.q.abs_()
    a.k[:, ::3] = t.finfo(a.k.dtype).min if kv == "f16" else -1e30
    a.v[:, ::3] = t.finfo(a.v.dtype).max if kv == "f16" else 1e30
    a.check()


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_attn_eight_heads_of_not_finite_values_that_are_seen(kv, dim):
    """As the formulas say, in the warps that see them and no others."""
    t = torch()
    a = Attn(kv, [899, 899, 899, 30], 16, 2, dim, 900, acc=True, seed=8)
    a.q.abs_()
    clean = a.want()
    a.k[0, 450, :dim] = math.nan            # K/V head 0 of row 0
    a.k[1, 460, dim:] = -math.inf           # head 1 of row 1: drops out
    a.v[2, 10, 3] = math.inf                # one value of head 0 of row 2
    a.k[3, 31:], a.v[3, 31:] = math.nan, math.inf     # behind the last entry
    acc0 = a.acc.clone()
    kd, vd = a.k.cpu().double().numpy(), a.v.cpu().double().numpy()
    kd[1, 460, dim:] = -1e30                # what -inf means where q is above 0
    vd[3, 31:], kd[3, 31:] = 0, 0
    a.call()
    got, acc = a.out.cpu().double().numpy(), a.acc.cpu().double().numpy()
    half = 8 * dim
    assert np.isnan(got[0, :half]).all() and np.isnan(acc[0, 0]).all()
    assert np.all(np.abs(got[0, half:] - clean[0][0, half:]) <= clean[1][0, half:])
    want, tol, want_acc, acc_tol = ref.attn(a.q.cpu().double().numpy()[1:2], kd[1:2], vd[1:2], [899], 16, 2, -1, 0,
                                            dim ** -0.5, acc0.cpu().double().numpy()[1:2])
    # (the tolerance's largest |q k| without the entry that drops out)
    assert np.all(np.abs(got[1] - want[0]) <= clean[1][1] * 2)
    assert np.all(np.abs(acc[1] - want_acc[0]) <= clean[3][1] * 2)
    seen = np.arange(16 * dim) % dim == 3
    seen[half:] = False
    assert np.isposinf(got[2, seen]).all()
    assert np.all(np.abs(got[2, ~seen] - clean[0][2, ~seen]) <= clean[1][2, ~seen])
    assert np.all(np.abs(got[3] - clean[0][3]) <= clean[1][3])
    no_error()


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [136, 160, 192, 200, 248, 256])
@pytest.mark.parametrize("group,n", [(5, 17), (6, 1), (7, 64), (8, 300), (16, 65), (8, 4000)])
def test_attn_eight_long_heads_of_16_bit_caches(kv, dim, group, n):
    """Two warps share V's values: heads padded to whole steps, entries to whole stages."""
    Attn(kv, [n - 1, n // 2, n // 3], 2 * group, 2, dim, n, window=n // 2 + 20, sinks=2, seed=dim + n).check()


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [136, 192, 256])
def test_attn_eight_long_heads_of_not_finite_values_that_are_seen(kv, dim):
    test_attn_eight_heads_of_not_finite_values_that_are_seen(kv, dim)


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("at", [0, 127, 128, 199])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attn_one_value_of_v_not_finite_in_either_half(kv, at, bad):
    """It reaches its own output only, whichever of the two warps holds it."""
    t = torch()
    a = Attn(kv, [499, 250], 16, 2, 200, 500, seed=at)
    a.v[0, 77, at] = bad
    want = a.want()
    a.call()
    got, w, tol = a.out.cpu().double().numpy(), *want[:2]
    hit = np.zeros_like(w, dtype=bool)
    hit[0, [g * 200 + at for g in range(8)]] = True
    assert not np.isfinite(got[hit]).any() and not np.isfinite(w[hit]).any()
    assert np.all(np.abs(got[~hit] - w[~hit]) <= tol[~hit])
    assert np.all(np.abs(a.acc.cpu().double().numpy() - want[2]) <= want[3])
    no_error()


@pytest.mark.parametrize("heads,kv_heads,dim", [(1024, 4, 16), (128, 1, 64), (1024, 1024, 8), (71, 71, 128)])
def test_attn_many_heads(heads, kv_heads, dim):
    Attn("bf16", [90, 12], heads, kv_heads, dim, 91, window=60, sinks=1, seed=heads).check()


@pytest.mark.parametrize("rows", [1, 3, 40, 256])
def test_attn_ragged_batches(rows):
    pos = [(37 * i * i + 11) % 400 - 1 for i in range(rows)]
    Attn("f16", pos, 8, 2, 64, 400, window=150, sinks=5, seed=rows, pad=5).check()


@pytest.mark.parametrize("kv,heads,dim,n", [
    ("f32", 8, 256, 9000), ("f32", 8, 72, 20000), ("f32", 5, 8, 30000), ("f32", 1, 64, 60000), ("f32", 1, 8, 70000),
    ("f32", 2, 200, 20000), ("bf16", 8, 128, 30000), ("bf16", 3, 24, 60000), ("bf16", 1, 256, 40000),
    ("f16", 7, 40, 30000), ("f16", 4, 200, 20000), ("f16", 6, 256, 15000)])
def test_attn_one_head_cut_in_many_parts(kv, heads, dim, n):
    """More parts of a K/V head than are joined at a time, of few values and of many."""
    Attn(kv, [n - 1], heads, 1, dim, n, seed=n + dim).check()
    Attn(kv, [n - 1, n // 9], heads, 1, dim, n, window=n // 2, sinks=5, seed=n - dim).check()


def test_attn_strided_rows():
    a = Attn("bf16", [50, 20, 63], 6, 3, 24, 64, seed=5, pad=13)
    a.check()
    assert bool((a.wide_out[:, 6 * 24:] == 7.0).all())      # what lies behind the rows is left alone


def test_attn_large_scores_and_scale():
    # scores of some hundreds: one weight near 1, the others next to nothing
    Attn("f32", [120], 4, 1, 64, 121, spread=40.0, seed=3).check()
    Attn("f32", [120], 4, 1, 64, 121, seed=4).check(scale=-0.7)
    Attn("f32", [120], 4, 1, 64, 121, seed=4).check(scale=0.0)


def test_attn_growing_scores():
    """Every entry's score above the last one's: the running maximum moves at each step."""
    a = Attn("f32", [699], 4, 1, 64, 700, seed=9)
    t = torch()
    a.k[:] = t.arange(700, device="cuda")[None, :, None] * 0.25
    a.q[:] = 0.5
    a.check()


@pytest.mark.parametrize("kv", ["f32", "f16", "bf16"])
def test_attn_masked_entries_do_not_matter(kv):
    pos, window, sinks = [40, 299, 150, -1], 64, 3
    clean = Attn(kv, pos, 8, 2, 64, 300, window=window, sinks=sinks, seed=1)
    dirty = Attn(kv, pos, 8, 2, 64, 300, window=window, sinks=sinks, seed=1)
    for m, p in enumerate(pos):
        see = set(ref.visible(p, window, sinks))
        for i in range(300):
            if i not in see:
                dirty.k[m, i] = (math.nan, math.inf, -math.inf)[i % 3]
                dirty.v[m, i] = (math.inf, math.nan, -math.inf)[i % 3]
    clean.check()
    dirty.call()
    assert torch().equal(clean.out, dirty.out) and torch().equal(clean.acc, dirty.acc)
    no_error()


def test_attn_empty_rows():
    a = Attn("f32", [-1, 5, -1], 4, 2, 32, 10, seed=2)
    before = a.acc.clone()
    a.check()
    assert bool((a.out[0] == 0).all()) and bool((a.out[2] == 0).all())
    assert torch().equal(a.acc[0], before[0])
    b = Attn("f32", [9, 0], 4, 2, 32, 10, window=0, sinks=0, seed=2)
    b.check()
    assert bool((b.out == 0).all())


def test_attn_position_out_of_range():
    t = torch()
    a = Attn("f32", [5, 5, 5, 5], 4, 2, 32, 10, seed=2)
    a.posd = t.tensor([5, 10, -2, 2 ** 31 - 1], dtype=t.int32, device="cuda")
    before = a.acc.clone()
    want = a.want()[0]
    a.call()
    assert native.q8_device_error() == 2
    assert np.allclose(a.out[0].cpu().numpy(), want[0], rtol=0, atol=1e-5)
    assert bool((a.out[1:] == 0).all()) and t.equal(a.acc[1:], before[1:])
    no_error()


def test_attn_not_finite_values_that_are_seen():
    """A NaN key makes its K/V head's rows NaN, a key of -inf scores drops out, as the formulas say."""
    t = torch()
    a = Attn("f32", [99, 99], 4, 2, 32, 100, acc=False, seed=8)
    a.q.abs_()
    a.k[0, 50, :32] = math.nan          # head 0 of row 0
    a.k[1, 60, 32:] = -math.inf         # head 1 of row 1
    want = a.want()[0]
    a.call()
    got = a.out.cpu().numpy()
    assert np.isnan(got[0, :64]).all() and not np.isnan(got[0, 64:]).any()
    assert np.allclose(got[1], want[1], rtol=1e-4, atol=1e-5)
    a.v[1, 10, 0] = math.inf            # a weight above 0 times infinity, in one value of head 0
    a.call()
    got = a.out.cpu().numpy()
    assert np.isposinf(got[1, 0]) and np.isposinf(got[1, 32]) and np.isfinite(got[1, 1:32]).all()
    no_error()


def test_attn_every_score_minus_infinity_is_nan():
    a = Attn("f32", [20], 2, 1, 32, 21, acc=False, seed=8)
    a.q.abs_()
    a.k.fill_(-math.inf)
    a.call()
    assert bool(a.out.isnan().all())


def test_attn_repeats_bit_for_bit():
    a = Attn("bf16", [3000, 7, 1500], 8, 2, 128, 3001, seed=6)
    start = a.acc.clone()
    a.call()
    out, acc = a.out.clone(), a.acc.clone()
    for _ in range(5):
        a.acc.copy_(start)
        a.call()
        assert torch().equal(a.out, out) and torch().equal(a.acc, acc)


def test_attn_one_workspace_for_calls_of_other_sizes():
    t = torch()
    calls = [Attn("f32", [900, 20], 8, 2, 64, 901, seed=1), Attn("f16", [100] * 30, 6, 6, 32, 101, seed=2),
             Attn("bf16", [2000], 16, 1, 128, 2001, window=700, sinks=1, seed=3)]
    size = max(c.ws.numel() for c in calls)
    ws = t.zeros(size, dtype=t.uint8, device="cuda")
    for c in calls + calls[::-1]:
        c.ws = ws
        c.check()


def test_one_workspace_for_attention_eviction_and_head():
    """The three calls whose workspace may be one buffer, in turn, several times."""
    t = torch()
    from q8_quantized_projection_gb300 import synth
    a = Attn("f16", [3000, 100, 2500], 8, 2, 64, 3001, seed=1)
    e = Evict("f32", [799, 300], 3, 32, 800, 400, sinks=2, recent=9, seed=2)
    rows, n, k = 3, 4096, 1024
    rng = synth.rng_for(5)
    q, s = synth.q8_weights(rng, n, k)
    qd, sd = t.from_numpy(q).cuda(), t.from_numpy(s.view(np.int16)).cuda()
    xq, xd = native.activation_buffers("i8", rows, k)
    native.act_quant("i8", t.randn(rows, k, device="cuda"), xq, xd)
    y = t.empty(rows, n, device="cuda")
    native.q8_proj("i8", qd, sd, xq, xd, rows, y)
    size = max(a.ws.numel(), e.ws.numel(), native.head_argmax_workspace(rows))
    ws = t.zeros(size, dtype=t.uint8, device="cuda")
    a.ws = e.ws = ws
    tok = t.empty(rows, dtype=t.int32, device="cuda")
    for _ in range(3):
        a.check()
        e.posd.copy_(t.tensor(e.pos, dtype=t.int32))
        e.check()
        tok.fill_(-1)
        native.head_argmax("i8", qd, sd, xq, xd, rows, tok, ws)
        assert t.equal(tok.long(), y.argmax(1))


def test_attn_offsets_past_32_bits():
    """The second row's entries lie past 2^31 values and 2^32 bytes."""
    t = torch()
    n_pos, dim = (1 << 23) + 5, 256
    k = t.empty(2, n_pos, dim, dtype=t.float16, device="cuda")
    v = t.empty(2, n_pos, dim, dtype=t.float16, device="cuda")
    g = t.Generator(device="cuda").manual_seed(1)
    window, sinks, rows = 50, 2, 2
    see = [0, 1] + list(range(n_pos - 50, n_pos))
    small_k = t.randn(2, 52, dim, device="cuda", generator=g).half()
    small_v = t.randn(2, 52, dim, device="cuda", generator=g).half()
    k[:, see], v[:, see] = small_k, small_v
    q = t.randn(rows, 2 * dim, device="cuda", generator=g)
    out = t.empty(rows, 2 * dim, device="cuda")
    acc = t.zeros(rows, 1, n_pos, device="cuda")
    pos = t.tensor([n_pos - 1] * 2, dtype=t.int32, device="cuda")
    native.attn_decode(q, k, v, pos, out, native.attn_workspace(rows, 2, 1, dim, n_pos, window, sinks, True), 2, 1,
                       window=window, sinks=sinks, acc=acc)
    f = lambda x: x.cpu().double().numpy()  # noqa: E731
    want, tol, want_acc, acc_tol = ref.attn(f(q), f(small_k), f(small_v), [51, 51], 2, 1, -1, 0, dim ** -0.5,
                                            np.zeros((2, 1, 52)))
    assert np.all(np.abs(f(out) - want) <= tol)
    assert np.all(np.abs(f(acc[:, :, see]) - want_acc) <= acc_tol)
    assert float(acc.sum()) == pytest.approx(4.0, rel=1e-4)
    no_error()


@pytest.mark.parametrize("kv,heads", [("f16", 1024), ("f32", 1024)])
def test_attn_tiles_of_several_stages(kv, heads):
    """So many heads over so long a cache that a tile holds several stages (its count stays below 2^31)."""
    t = torch()
    n_pos, n, dim = (1 << 28) + 3, 3001, 8
    k = t.empty(1, n_pos, dim, dtype=dt(kv), device="cuda")
    v = t.empty(1, n_pos, dim, dtype=dt(kv), device="cuda")
    g = t.Generator(device="cuda").manual_seed(1)
    k[:, :n], v[:, :n] = (t.randn(1, n, dim, device="cuda", generator=g).to(dt(kv)) for _ in range(2))
    q = t.randn(1, heads * dim, device="cuda", generator=g)
    out = t.empty(1, heads * dim, device="cuda")
    native.attn_decode(q, k, v, t.tensor([n - 1], dtype=t.int32, device="cuda"), out,
                       native.attn_workspace(1, heads, 1, dim, n_pos), heads, 1)
    f = lambda x: x.cpu().double().numpy()  # noqa: E731
    want, tol, _, _ = ref.attn(f(q), f(k[:, :n]), f(v[:, :n]), [n - 1], heads, 1, -1, 0, dim ** -0.5)
    assert np.all(np.abs(f(out) - want) <= tol)
    no_error()


# ---------------------------------------------------------------- kv_evict

class Evict:
    def __init__(self, kv, pos, kv_heads, dim, n_pos, budget, sinks=0, recent=0, seed=0, acc=None):
        t = torch()
        g = t.Generator(device="cuda").manual_seed(seed)
        rows = len(pos)
        self.kv_heads, self.dim, self.n_pos, self.pos = kv_heads, dim, n_pos, pos
        self.budget, self.sinks, self.recent = budget, sinks, recent
        self.k = t.randn(rows, n_pos, kv_heads * dim, device="cuda", generator=g).to(dt(kv))
        self.v = t.randn(rows, n_pos, kv_heads * dim, device="cuda", generator=g).to(dt(kv))
        self.posd = t.tensor(pos, dtype=t.int32, device="cuda")
        a = t.randn(rows, kv_heads, n_pos, device="cuda", generator=g).exp()
        self.acc = t.where(a < 0.3, 0.0, a) if acc is None else acc     # many ties at zero
        self.kept = t.full((rows, kv_heads, budget), -7, dtype=t.int32, device="cuda")
        self.ws = t.randint(0, 255, (native.kv_evict_workspace(rows, kv_heads, budget),), dtype=t.uint8,
                            device="cuda", generator=g)

    def call(self, new_pos, new_acc, kept, stream=None):
        native.kv_evict(self.k, self.v, self.posd, self.acc, new_pos, new_acc, self.ws, self.kv_heads, self.budget,
                        sinks=self.sinks, recent=self.recent, kept=kept, stream=stream)

    def check(self, in_place=False):
        t = torch()
        bits = lambda x: x.view(t.int16 if x.dtype != t.float32 else t.int32).cpu().numpy()  # noqa: E731
        want = ref.evict(bits(self.k), bits(self.v), self.pos, self.acc.cpu().numpy(), self.kv_heads, self.budget,
                         self.sinks, self.recent, self.n_pos)
        if in_place:
            new_pos, new_acc = self.posd, self.acc
        else:
            new_pos, new_acc = t.full_like(self.posd, -9), t.full_like(self.acc, -9.0)
        self.call(new_pos, new_acc, None if in_place else self.kept)
        assert np.array_equal(bits(self.k), want[0]) and np.array_equal(bits(self.v), want[1])
        assert np.array_equal(new_pos.cpu().numpy(), want[2])
        assert np.array_equal(new_acc.cpu().numpy().view(np.uint32), want[3].view(np.uint32))
        if not in_place:
            assert np.array_equal(self.kept.cpu().numpy(), want[4])
        no_error()


@pytest.mark.parametrize("kv", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 24, 64, 80, 128, 200, 256])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_types_and_dims(kv, dim, in_place):
    Evict(kv, [199, 100, 99, -1, 130], 3, dim, 200, 100, sinks=4, recent=10, seed=dim).check(in_place)


@pytest.mark.parametrize("n,budget,sinks,recent", [
    (2, 1, 0, 0), (2, 1, 1, 0), (2, 1, 0, 1), (50, 1, 0, 0), (50, 49, 0, 0), (50, 49, 20, 29), (50, 10, 10, 0),
    (50, 10, 0, 10), (50, 10, 4, 6), (300, 257, 1, 1), (1025, 1024, 4, 64), (5000, 33, 1, 2), (3000, 2999, 0, 1),
    (4097, 2048, 4, 1000), (9000, 4100, 0, 0)])
def test_evict_sizes(n, budget, sinks, recent):
    Evict("bf16", [n - 1], 2, 32, n + 3, budget, sinks, recent, seed=n).check()
    Evict("f32", [n - 1], 1, 16, n, budget, sinks, recent, seed=n + 1).check(in_place=True)


@pytest.mark.parametrize("n,budget,sinks,recent", [
    (8193, 4000, 4, 100), (9000, 100, 60, 40), (20000, 19999, 0, 0), (40001, 33, 3, 30), (66000, 30000, 4, 2000),
    (70001, 69000, 100, 1), (131073, 1, 0, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_rows(n, budget, sinks, recent, in_place):
    """Selections on several CTAs and past what their lanes hold, walks of clusters."""
    Evict("bf16", [n - 1, n // 2], 1, 8, n, budget, sinks, recent, seed=n).check(in_place)


@pytest.mark.parametrize("kv,rows,heads,dim,n,budget", [
    ("f16", 1, 8, 256, 9000, 7000), ("f32", 3, 2, 128, 12000, 5000), ("bf16", 2, 8, 80, 8000, 6501),
    ("f32", 1, 8, 24, 9000, 4000), ("bf16", 1, 2, 200, 20000, 12345)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_walks_of_clusters(kv, rows, heads, dim, n, budget, in_place):
    """Few slices, narrow and wide ones, whose clusters walk together."""
    Evict(kv, [n - 1 - 700 * m for m in range(rows)], heads, dim, n, budget, 4, 900, seed=n + dim).check(in_place)


def test_evict_rows_at_most_the_budget_stay():
    e = Evict("f32", [9, 0, -1, 5], 2, 16, 12, 10, sinks=2, recent=2)
    k = e.k.clone()
    e.check()
    assert torch().equal(e.k, k)


@pytest.mark.parametrize("what", ["zero", "same", "nan", "inf", "negative", "denormal", "rising", "falling", "high"])
def test_evict_weights(what):
    t = torch()
    n = 700
    a = t.rand(2, 2, n, device="cuda", generator=t.Generator(device="cuda").manual_seed(4))
    i = t.arange(n, device="cuda")
    a = {"zero": t.where(i % 2 == 0, 0.0, -0.0).expand(2, 2, n).contiguous(),
         "same": t.full_like(a, 0.125), "nan": t.where(i % 3 == 0, math.nan, a),
         "inf": t.where(i % 5 == 0, math.inf, t.where(i % 7 == 0, -math.inf, a)), "negative": a - 0.5,
         "denormal": a * 1e-39, "rising": (i * 1e-3).expand(2, 2, n).contiguous(),
         "falling": (-i * 1e-3).expand(2, 2, n).contiguous(),
         # keys that differ in their last bits only
         "high": (1.0 + (i * 37 % 64) * 2.0 ** -23).expand(2, 2, n).contiguous()}[what]
    Evict("f16", [n - 1, n - 40], 2, 16, n, 300, sinks=3, recent=20, acc=a.clone()).check()
    Evict("f16", [n - 1, n - 40], 2, 16, n, 600, sinks=0, recent=0, acc=a.clone()).check(in_place=True)


@pytest.mark.parametrize("n,budget", [(300, 140), (2049, 1000), (3900, 3001), (6000, 2500), (30000, 9000)])
@pytest.mark.parametrize("levels", [1, 3, 40])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_ties_at_every_length(n, budget, levels, in_place):
    """Weights of few values: the last place falls among equals, of which the first ones stay."""
    e = Evict("f16", [n - 1, n - 2], 40 if n < 400 else 2, 8, n, budget, sinks=3, recent=20, seed=n)
    e.acc.mul_(levels).floor_().div_(levels)
    e.check(in_place)


def test_evict_position_out_of_range():
    t = torch()
    e = Evict("f32", [11, 11, 11], 2, 16, 12, 6)
    e.posd = t.tensor([12, -2, 2 ** 31 - 1], dtype=t.int32, device="cuda")
    k, v = e.k.clone(), e.v.clone()
    new_pos, new_acc = t.zeros_like(e.posd), t.zeros_like(e.acc)
    e.call(new_pos, new_acc, e.kept)
    assert native.q8_device_error() == 2
    assert t.equal(e.k, k) and t.equal(e.v, v) and t.equal(new_pos, e.posd) and t.equal(new_acc, e.acc)
    assert bool((e.kept == -1).all())


def test_evict_large_batch():
    pos = [(97 * i + 300) % 1100 for i in range(96)]
    Evict("bf16", pos, 8, 64, 1100, 500, sinks=4, recent=100, seed=12).check()


def test_evict_offsets_past_32_bits():
    t = torch()
    n_pos, dim, budget = (1 << 23) + 5, 256, 64
    k = t.zeros(2, n_pos, dim, dtype=t.float16, device="cuda")
    v = t.zeros(2, n_pos, dim, dtype=t.float16, device="cuda")
    acc = t.zeros(2, 1, n_pos, device="cuda")
    best = [n_pos - 10 - 131 * i for i in range(32)][::-1]
    acc[1, 0, best] = 1.0
    k[1, best] = t.arange(32, device="cuda", dtype=t.float16)[:, None] + 1
    v[1, best] = -(t.arange(32, device="cuda", dtype=t.float16)[:, None] + 1)
    pos = t.tensor([5, n_pos - 1], dtype=t.int32, device="cuda")
    ws = t.empty(native.kv_evict_workspace(2, 1, budget), dtype=t.uint8, device="cuda")
    kept = t.empty(2, 1, budget, dtype=t.int32, device="cuda")
    native.kv_evict(k, v, pos, acc, pos, acc, ws, 1, budget, sinks=32, kept=kept)
    assert pos.tolist() == [5, budget - 1] and kept[1, 0].tolist() == list(range(32)) + best
    assert bool((k[1, 32:64, 0] == t.arange(32, device="cuda") + 1).all())
    assert bool((v[1, 32:64, 255] == -(t.arange(32, device="cuda") + 1)).all())
    assert float(acc.sum()) == 32.0
    no_error()


# ------------------------------------------------------------- head_sample

def draw(x, u, t=None, k=None, p=None, mp=None):
    T = torch()
    rows = x.shape[0]
    col = lambda v, ty: None if v is None else T.tensor(v, dtype=ty, device="cuda")  # noqa: E731
    tok = T.full((rows,), -5, dtype=T.int32, device="cuda")
    prob, kept = T.full((rows,), -5.0, device="cuda"), T.full((rows,), -5, dtype=T.int32, device="cuda")
    native.head_sample(x, col(u, T.float32), tok, temperature=col(t, T.float32), top_k=col(k, T.int32),
                       top_p=col(p, T.float32), min_p=col(mp, T.float32), prob=prob, kept=kept)
    return tok.cpu().numpy(), prob.cpu().numpy(), kept.cpu().numpy()


def check_draw(x, u, t=None, k=None, p=None, mp=None):
    """Token and count as the 64-bit form's.  prob is w / S rounded to binary32
    (2^-24): w and each term of S carry at most 2^-29 of themselves, so their
    quotient 2^-28, and a term loses less than one unit of 2^-shift, shift = 62
    - ceil(log2 N), of the largest weight, which S is no less than: N 2^-shift."""
    n = x.shape[1]
    units = n * 2.0 ** ((n - 1).bit_length() - 62)
    got = draw(x, u, t, k, p, mp)
    f32 = lambda v, d: [d] * x.shape[0] if v is None else [float(np.float32(a)) for a in v]  # noqa: E731
    xs = x.cpu().numpy()
    for m, (uu, tt, pp, mm) in enumerate(zip(f32(u, 0), f32(t, 1.0), f32(p, 1.0), f32(mp, 0.0))):
        tok, prob, kept = ref.sample(xs[m], uu, tt, 0 if k is None else k[m], pp, mm)
        assert (got[0][m], got[2][m]) == (tok, kept), (m, got[0][m], got[2][m], tok, kept)
        assert abs(float(got[1][m]) - prob) <= prob * (2.0 ** -24 + 2.0 ** -28 + units) + 2.0 ** -149


def logits(rows, n, spread=2.0, seed=0, pad=0):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return (t.randn(rows, n + pad, device="cuda", generator=g) * spread)[:, :n]


@pytest.mark.parametrize("n", [1, 2, 3, 31, 33, 100, 511, 1000, 1025, 4097, 20001, 33333])
def test_sample_sizes(n):
    x = logits(6, n, seed=n)
    u = [0.0, 0.1, 0.5, 0.9, 0.9999, 0.33]
    check_draw(x, u)
    check_draw(x, u, t=[1.0, 0.5, 2.0, 0.0, 0.7, 1.3], k=[5, 1, 0, 7, 300, 50], p=[0.9, 1.0, 0.5, 0.2, 0.99, 0.0],
               mp=[0.0, 0.1, 0.01, 0.0, 0.3, 0.05])


@pytest.mark.parametrize("n,rows", [(128256, 2), (131073, 1), (262145, 1), (1 << 20, 1)])
def test_sample_large_vocabularies(n, rows):
    x = logits(rows, n, seed=n % 1000)
    check_draw(x, [0.7] * rows)
    check_draw(x, [0.37] * rows, t=[0.8] * rows, k=[1500] * rows, p=[0.9] * rows)
    check_draw(x, [0.91] * rows, p=[0.95] * rows, mp=[0.001] * rows)


@pytest.mark.parametrize("rows", [1, 5, 64, 256])
def test_sample_batches(rows):
    x = logits(rows, 3001, spread=3.0, seed=rows, pad=11)
    i = np.arange(rows)
    check_draw(x, list((i * 0.6180339) % 1.0), t=list(0.3 + (i % 5) * 0.4), k=list(map(int, (i % 4) * 23)),
               p=list(np.where(i % 3 == 0, 1.0, 0.5 + (i % 50) * 0.01)), mp=list((i % 6) * 0.02))


@pytest.mark.parametrize("n", [9001, 128256])
def test_sample_long_cuts(n):
    """Top-k past what one list holds, nuclei of nearly everything, and both."""
    x = logits(4, n, spread=1.5, seed=n % 13)
    u = [0.03, 0.4, 0.77, 0.98]
    check_draw(x, u, k=[2047, 2048, 2049, 5000])
    check_draw(x, u, p=[0.999, 0.9999, 0.99999, 1.0 - 2.0 ** -24])
    check_draw(x, u, k=[8000, 2500, 4000, 600], p=[0.9, 0.99, 0.5, 0.999], t=[1.0, 3.0, 0.4, 1.0])
    check_draw(x, u, k=[7000, 0, 3000, 0], mp=[0.01, 0.001, 1e-6, 1e-3], t=[1.0, 2.0, 5.0, 0.2])


def test_sample_few_levels():
    """Logits of few values (as 8-bit mantissas give): cuts fall among many ties."""
    x = (logits(6, 40000, spread=2.0, seed=2) * 4).round() / 4
    u = [0.1, 0.3, 0.5, 0.7, 0.9, 0.99]
    check_draw(x, u, k=[50, 1000, 5000, 20000, 1, 39999])
    check_draw(x, u, p=[0.1, 0.3, 0.5, 0.7, 0.9, 0.99])
    check_draw(x, u, k=[500, 3000, 0, 100, 30000, 10], p=[0.9, 0.5, 0.95, 0.99, 0.8, 0.3], mp=[0.0, 0.01, 0.1, 0.05, 0.0, 0.2])


@pytest.mark.parametrize("n", [1900, 15000, 40000])
@pytest.mark.parametrize("many", [60, 300, 1000, 2000])
@pytest.mark.parametrize("sort", [False, True])
def test_sample_cuts_among_equal_logits(n, many, sort):
    """Equal logits by tens to thousands where the cut falls, scattered and side by side."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(n + many)
    x = (t.rand(6, n, device="cuda", generator=g) * (n / many)).floor() * (4.0 * many / n)
    if sort:
        x = x.sort(dim=1, descending=True).values.contiguous()
    u = [0.0, 0.317, 0.513, 0.0, 0.913, 0.9917]
    p = [0.117, 0.317, 0.517, 0.717, 0.917, 0.9917]
    check_draw(x, u, p=p)
    check_draw(x, u, p=p, mp=[0.0, 0.1, 0.01, 0.2, 0.0, 0.3], t=[1.0, 2.0, 0.5, 1.5, 3.0, 1.0])
    check_draw(x, u, k=[1700, 1234, 1500, 1801, 1111, 1899], p=p)


@pytest.mark.parametrize("n", [2, 127, 128, 129, 6000, 128256])
@pytest.mark.parametrize("allowed", [1, 2, 17, 128, 129])
def test_sample_few_tokens_allowed(n, allowed):
    """A mask that leaves few tokens of a row, as a grammar does."""
    t = torch()
    x = logits(6, n, spread=2.5, seed=n + allowed)
    if allowed < n:
        order = t.rand(6, n, device="cuda", generator=t.Generator(device="cuda").manual_seed(n)).argsort(dim=1)
        x = x.scatter(1, order[:, allowed:], -math.inf).contiguous()
    u = [0.0, 0.21, 0.5, 0.77, 0.93, 0.9999]
    check_draw(x, u)
    check_draw(x, u, p=[0.3, 0.6, 0.9, 0.95, 0.99, 0.5], t=[1.0, 0.5, 2.0, 3.0, 0.7, 1.3])
    check_draw(x, u, k=[3, 0, 50, 127, 1, 128], p=[0.9, 0.8, 1.0, 0.7, 0.6, 0.99], mp=[0.0, 0.2, 0.05, 0.0, 0.1, 0.01])


def test_sample_shares_next_to_a_border():
    """Nuclei that end a few steps of binary32 beside a token's border, tokens far apart."""
    t = torch()
    x = t.full((24, 3000), -9.0, device="cuda")
    at = [(i * 251 + 7) % 3000 for i in range(24)]
    x[:, at] = t.arange(24, device="cuda") * -0.21 + 1.3
    w = np.exp(np.sort(x[0].cpu().double().numpy())[::-1] - 1.3)
    cum = w.cumsum() / w.sum()
    p = []
    for i in range(24):                     # 2 to 5 steps above or below the border of token i // 2
        v = np.float32(cum[i // 2])
        for _ in range(2 + i % 4):
            v = np.nextafter(v, np.float32(2 if i % 2 else 0), dtype=np.float32)
        p.append(float(v))
    check_draw(x, [0.5 + 0.02 * i for i in range(24)], p=p)


def test_sample_rows_masked_by_the_lowest_float():
    """Masks of -3.4e38 beside ordinary logits, and a row of nothing else."""
    t = torch()
    low = t.finfo(t.float32).min
    x = logits(5, 5000, seed=6)
    x[0, 10:] = low
    x[1, ::2] = low
    x[2, 1:] = low
    x[3] = low
    x[4, 100:4000] = -math.inf
    u = [0.5, 0.9, 0.3, 0.6, 0.999]
    for kw in (dict(), dict(k=[5, 100, 3, 7, 900]), dict(p=[0.9, 0.8, 0.5, 0.25, 0.95]), dict(mp=[0.1] * 5),
               dict(k=[2400] * 5, p=[0.7] * 5)):
        check_draw(x, u, **kw)


def test_sample_every_token_can_be_drawn():
    """Weights 1 : 2 : 4 (exact in logits of log 2 only to rounding): each number falls in its own share."""
    t = torch()
    x = t.log(t.tensor([[1.0, 2.0, 4.0, 1.0]], device="cuda")).repeat(8, 1)
    tok, prob, kept = draw(x, [0.0, 0.12, 0.13, 0.37, 0.38, 0.86, 0.88, 0.999])
    assert tok.tolist() == [0, 0, 1, 1, 2, 2, 3, 3] and kept.tolist() == [4] * 8
    assert np.allclose(prob, [0.125, 0.125, 0.25, 0.25, 0.5, 0.5, 0.125, 0.125], rtol=1e-6)


def test_sample_ties_go_to_the_lowest_index():
    t = torch()
    n = 3000
    x = t.zeros(5, n, device="cuda")
    u = [0.0, 0.5, 0.999, 0.5, 0.25]
    check_draw(x, u, k=[10, 10, 10, 0, 1])
    check_draw(x, u, p=[0.5, 0.25, 0.75, 0.125, 0.0])
    check_draw(x, u, t=[0.0] * 5)
    x[:, 1000:] = 1.0                       # the ties that count lie behind others
    check_draw(x, u, k=[10, 1500, 2000, 2500, 3000])
    x = (t.arange(n, device="cuda") % 7).float().repeat(5, 1)
    check_draw(x, u, k=[429, 430, 5, 900, 2999], p=[0.9, 1.0, 0.5, 0.77, 0.999])


def test_sample_masked_and_infinite_logits():
    t = torch()
    inf, nan = math.inf, math.nan
    x = logits(8, 500, seed=3)
    x[0, ::2] = -inf
    x[1, 5:] = -inf
    x[2, :499] = nan
    x[3, 100] = inf
    x[4, [7, 300, 450]] = inf
    x[5] = -inf
    x[6] = nan
    x[7, ::3] = nan
    u = [0.7, 0.99, 0.5, 0.5, 0.5, 0.5, 0.5, 0.2]
    for kw in (dict(), dict(k=[20] * 8), dict(p=[0.8] * 8), dict(mp=[0.1] * 8), dict(t=[0.0] * 8),
               dict(k=[400] * 8, p=[0.6] * 8, mp=[0.001] * 8, t=[1.5] * 8)):
        check_draw(x, u, **kw)
    no_error()
    z = t.tensor([[0.0, -0.0, -1.0, 0.0]], device="cuda")
    check_draw(z, [0.5], k=[2])


def test_sample_odd_settings():
    x = logits(6, 400, seed=8)
    u = [0.4] * 6
    check_draw(x, u, k=[-3, 400, 401, 2 ** 31 - 1, -2 ** 31, 399])
    check_draw(x, u, p=[-1.0, 0.0, 1e-30, 1.0, 7.0, math.inf])
    check_draw(x, u, mp=[-1.0, 0.0, 1.0, 1.5, math.inf, -math.inf])
    check_draw(x, u, t=[1e30, 100.0, 1e-3, 2.0 ** -60, 2.0 ** -61, math.inf])
    check_draw(x, [-1.0, math.nan, 1.0, 5.0, math.inf, -math.inf])
    big = x * 1e37
    check_draw(big, u, t=[1e38, 1e37, 1.0, 3e38, math.inf, 1e36])
    no_error()


def test_sample_refused_settings():
    x = logits(5, 100)
    nan = math.nan
    for kw in (dict(t=[1.0, -0.5, nan, 1.0, 1.0]), dict(p=[1.0, nan, nan, 1.0, 1.0]),
               dict(mp=[0.0, nan, nan, 0.0, 0.0])):
        check_draw(x, [0.5] * 5, **kw)
        assert native.q8_device_error() == 3
    no_error()


def test_sample_follows_its_distribution():
    """4096 evenly spaced numbers: each token's share is its probability to one step at each end."""
    x = logits(1, 50, spread=1.0, seed=5)
    n = 4096
    tok = np.concatenate([draw(x.repeat(256, 1), list((np.arange(256) + 256 * b + 0.5) / n))[0]
                          for b in range(n // 256)])
    w = np.exp(x[0].cpu().double().numpy())
    assert np.all(np.abs(np.bincount(tok, minlength=50) - n * w / w.sum()) <= 1.0 + 1e-6)


# ---------------------------------------------------- streams, graphs, a step

def test_calls_on_another_stream_and_in_a_graph():
    t = torch()
    a = Attn("f32", [500, 30, 210], 8, 2, 64, 512, window=300, sinks=2, seed=11)
    e = Evict("f32", [511, 100, 400], 2, 64, 512, 256, sinks=2, recent=30, seed=12)
    x = logits(3, 1000, seed=13)
    u = t.tensor([0.2, 0.5, 0.8], device="cuda")
    tok = t.zeros(3, dtype=t.int32, device="cuda")
    k0, v0, acc0 = e.k.clone(), e.v.clone(), a.acc.clone()
    new_pos, new_acc = t.zeros_like(e.posd), t.zeros_like(e.acc)
    s = t.cuda.Stream()

    def step(stream=None):
        a.call(stream)
        e.call(new_pos, new_acc, e.kept, stream)
        native.head_sample(x, u, tok, stream=stream)

    def results():
        return [r.clone() for r in (a.out, a.acc, e.k, e.v, new_pos, new_acc, e.kept, tok)]

    step()
    want = results()
    t.cuda.synchronize()
    for how in ("stream", "graph"):
        if how == "graph":
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph, stream=s):
                step(s)
        for _ in range(2):
            a.out.zero_(), a.acc.copy_(acc0), e.k.copy_(k0), e.v.copy_(v0), e.kept.zero_(), tok.zero_()
            new_pos.zero_(), new_acc.zero_()
            t.cuda.synchronize()
            if how == "graph":
                graph.replay()
            else:
                step(s)
            t.cuda.synchronize()
            assert all(t.equal(g, w) for g, w in zip(results(), want)), how
    # a captured step follows the positions that its device memory holds
    a.posd.copy_(t.tensor([80, 511, 0], dtype=t.int32))
    a.pos = [80, 511, 0]
    a.acc.copy_(acc0)
    want = a.want()
    e.k.copy_(k0), e.v.copy_(v0)
    graph.replay()
    t.cuda.synchronize()
    assert np.all(np.abs(a.out.cpu().double().numpy() - want[0]) <= want[1])
    no_error()


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
def test_decode_steps_together(mode):
    """Some decode steps as a program runs them, captured into one graph: the fused QKV projection
    writes the caches, attention reads them and accumulates, a full cache is evicted, the head's
    logits are sampled.  Each operator is held to its 64-bit form on what the step gave it."""
    from q8_quantized_projection_gb300 import synth
    t = torch()
    rows, heads, kv_heads, dim, n_pos, budget, vocab, hidden = 3, 8, 2, 64, 24, 16, 1500, 1024
    sinks, recent, window = 2, 6, 14
    kv_dim, width = kv_heads * dim, (heads + 2 * kv_heads) * dim
    rng = synth.rng_for(3)
    put = lambda w: (t.from_numpy(w[0]).cuda(), t.from_numpy(w[1].view(np.int16)).cuda())  # noqa: E731
    wqkv, whead = put(synth.q8_weights(rng, width, hidden)), put(synth.q8_weights(rng, vocab, hidden))
    g = t.Generator(device="cuda").manual_seed(1)
    h = t.empty(rows, hidden, device="cuda")
    y, out = t.empty(rows, width, device="cuda"), t.empty(rows, heads * dim, device="cuda")
    logit, u = t.empty(rows, vocab, device="cuda"), t.empty(rows, device="cuda")
    k = t.full((rows, n_pos, kv_dim), math.nan, device="cuda")       # nothing may read what was never written
    v = t.full((rows, n_pos, kv_dim), math.nan, device="cuda")
    acc = t.zeros(rows, kv_heads, n_pos, device="cuda")
    pos = t.tensor([-1, 5, 14], dtype=t.int32, device="cuda")
    for m in range(rows):
        n = int(pos[m]) + 1
        k[m, :n], v[m, :n] = (t.randn(n, kv_dim, device="cuda", generator=g) for _ in range(2))
    tok = t.zeros(rows, dtype=t.int32, device="cuda")
    kept = t.zeros(rows, dtype=t.int32, device="cuda")
    ws = t.empty(native.q8_proj_fused_workspace(mode, rows, hidden), dtype=t.uint8, device="cuda")
    xq, xd = native.activation_buffers(mode, rows, hidden)
    aws = native.attn_workspace(rows, heads, kv_heads, dim, n_pos, window, sinks, True)
    top_p, temp = t.full((rows,), 0.9, device="cuda"), t.full((rows,), 0.8, device="cuda")

    def step():
        pos.add_(1)
        native.q8_proj_fused_kv(mode, *wqkv, h, y, ws, pos, heads * dim, k, v)
        native.attn_decode(y, k, v, pos, out, aws, heads, kv_heads, window=window, sinks=sinks, acc=acc)
        native.act_quant(mode, h, xq, xd, norm=True)
        native.q8_proj(mode, *whead, xq, xd, rows, logit)
        native.head_sample(logit, u, tok, temperature=temp, top_p=top_p, kept=kept)

    def shorten():
        ews = t.empty(native.kv_evict_workspace(rows, kv_heads, budget), dtype=t.uint8, device="cuda")
        native.kv_evict(k, v, pos, acc, pos, acc, ews, kv_heads, budget, sinks=sinks, recent=recent)

    f = lambda a: a.cpu().double().numpy()  # noqa: E731
    graph = None
    for i in range(20):
        h.normal_(generator=g)
        u.uniform_(generator=g)
        before = [pos.clone(), acc.clone(), k.clone(), v.clone()]
        if i == 1:
            graph = t.cuda.CUDAGraph()
            state = [b.clone() for b in before]
            with t.cuda.graph(graph):
                step()
            for dst, src in zip((pos, acc, k, v), state):
                dst.copy_(src)
        if graph is None:
            step()
        else:
            graph.replay()
        t.cuda.synchronize()
        at = pos.tolist()
        assert at == [p + 1 for p in before[0].tolist()]
        for m in range(rows):       # only the new entry of each cache changed
            now, old = k[m].clone(), before[2][m].clone()
            assert t.equal(now[at[m]], y[m, heads * dim:heads * dim + kv_dim])
            now[at[m]], old[at[m]] = 0, 0
            assert t.equal(now.nan_to_num(7.0), old.nan_to_num(7.0))
        kd, vd = f(k), f(v)
        for m in range(rows):
            kd[m, at[m] + 1:], vd[m, at[m] + 1:] = 0, 0
        want, tol, want_acc, acc_tol = ref.attn(f(y[:, :heads * dim]), kd, vd, at, heads, kv_heads, window, sinks,
                                                dim ** -0.5, f(before[1]))
        assert np.all(np.abs(f(out) - want) <= tol)
        assert np.all(np.abs(f(acc) - want_acc) <= acc_tol)
        for m in range(rows):
            assert (int(tok[m]), int(kept[m])) == ref.sample(f(logit[m]), float(u[m]), float(np.float32(0.8)), 0,
                                                              float(np.float32(0.9)))[::2]
        if max(at) == n_pos - 1:
            bits = lambda x: x.view(t.int32).cpu().numpy()  # noqa: E731
            want = ref.evict(bits(k), bits(v), at, acc.cpu().numpy(), kv_heads, budget, sinks, recent, n_pos)
            shorten()
            assert np.array_equal(bits(k), want[0]) and np.array_equal(bits(v), want[1])
            assert pos.tolist() == want[2].tolist() and np.array_equal(acc.cpu().numpy(), want[3])
    no_error()


def test_calls_at_once_on_two_streams():
    """Calls that overlap, each with its own buffers and workspace, give what they give alone."""
    t = torch()
    a = [Attn("bf16", [2500, 900, 4000], 8, 2, 128, 4001, seed=i) for i in range(2)]
    e = [Evict("f32", [1999, 700], 4, 64, 2000, 900, sinks=1, recent=50, seed=i) for i in range(2)]
    x = [logits(20, 5000, seed=i) for i in range(2)]
    u = t.rand(20, device="cuda", generator=t.Generator(device="cuda").manual_seed(3))
    tok = [t.zeros(20, dtype=t.int32, device="cuda") for _ in range(2)]
    top_p = t.full((20,), 0.8, device="cuda")
    start = [[v.clone() for v in (a[i].acc, e[i].k, e[i].v)] for i in range(2)]
    new = [(t.zeros_like(e[i].posd), t.zeros_like(e[i].acc)) for i in range(2)]

    def reset():
        for i in range(2):
            for dst, src in zip((a[i].acc, e[i].k, e[i].v), start[i]):
                dst.copy_(src)

    def call(i, stream=None):
        a[i].call(stream)
        e[i].call(*new[i], e[i].kept, stream)
        native.head_sample(x[i], u, tok[i], top_p=top_p, stream=stream)

    def results(i):
        return [v.clone() for v in (a[i].out, a[i].acc, e[i].k, e[i].v, *new[i], e[i].kept, tok[i])]

    want = []
    for i in range(2):
        call(i)
        want.append(results(i))
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(5):
        reset()
        t.cuda.synchronize()
        for i in range(2):
            call(i, streams[i])
        t.cuda.synchronize()
        for i in range(2):
            assert all(t.equal(g, w) for g, w in zip(results(i), want[i]))
    no_error()


def test_binding_checks():
    t = torch()
    a = Attn("f32", [5, 3], 4, 2, 32, 8, seed=1)

    def bad(error, **over):
        args = dict(q=a.q, k_cache=a.k, v_cache=a.v, pos=a.posd, out=a.out, workspace=a.ws, heads=4, kv_heads=2,
                    acc=a.acc)
        args.update(over)
        with pytest.raises(error):
            native.attn_decode(**args)

    bad(TypeError, q=a.q.half())
    bad(TypeError, k_cache=a.k.double(), v_cache=a.v.double())
    bad(TypeError, v_cache=a.v.half())
    bad(TypeError, pos=a.posd.long())
    bad(ValueError, pos=a.posd[:1])
    bad(ValueError, k_cache=a.k[:, :4])
    bad(ValueError, acc=a.acc[:, :1])
    bad(ValueError, heads=5)
    bad(ValueError, kv_heads=3)
    bad(ValueError, q=a.q.t().contiguous().t())
    bad(ValueError, workspace=a.ws.cpu())
    bad(ValueError, out=a.out.cpu())
    bad(native.Q8Error, out=a.q)
    bad(native.Q8Error, workspace=a.ws[:64])
    e = Evict("f32", [5, 3], 2, 16, 8, 4)
    with pytest.raises(ValueError):
        e.call(e.posd, e.acc, e.kept[:, :, :2])
    with pytest.raises(native.Q8Error):
        e.call(e.posd, e.acc.view(-1)[:e.acc.numel()].view_as(e.acc), e.kept) or \
            native.kv_evict(e.k, e.k, e.posd, e.acc, e.posd, e.acc, e.ws, 2, 4)
    x = logits(2, 10)
    with pytest.raises(TypeError):
        native.head_sample(x, t.zeros(2, device="cuda"), t.zeros(2, dtype=t.int64, device="cuda"))
    with pytest.raises(ValueError):
        native.head_sample(x, t.zeros(3, device="cuda"), t.zeros(2, dtype=t.int32, device="cuda"))
