"""Host-side checks of the quantised K/V caches' calls: what they refuse, before anything
touches a GPU, and their workspaces' sizes."""
import ctypes as C
import os
import subprocess
import sys

import pytest

from q8_quantized_projection_gb300 import build, native


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def P(n):
    """A 16-byte aligned placeholder pointer (never dereferenced), far from P of another n."""
    return C.c_void_p((n + 1) << 32)


K, V, POS, LENS, KC, KW, VC, VW, Q, OUT, ACC, WS, NPOS, NACC, KEPT = (P(i) for i in range(15))
BIG = 1 << 40


def off(p, n):
    return C.c_void_p(p.value + n)


def store(lib, **over):
    a = dict(k=K, v=V, src=0, ld_row=640, ld_tok=64, rows=2, T=10, kv_heads=2, dim=32, pos=POS, lens=LENS, kind=1,
             kc=KC, kw=KW, vc=VC, vw=VW, n_pos=64, stream=None)
    a.update(over)
    return lib.kvq_store(*a.values())


def load(lib, **over):
    a = dict(kind=1, kc=KC, kw=KW, vc=VC, vw=VW, rows=2, n_pos=64, kv_heads=2, dim=32, pos=POS, T=10, lens=LENS, dst=0,
             k=K, v=V, ld_row=640, ld_tok=64, stream=None)
    a.update(over)
    return lib.kvq_load(*a.values())


SIZES = [
    (dict(kind=2), 4), (dict(kind=-1), 4), (dict(rows=0), 2), (dict(rows=257), 2), (dict(n_pos=0), 2),
    (dict(n_pos=1 << 31), 2), (dict(kv_heads=0), 2), (dict(kv_heads=1025), 2), (dict(kv_heads=1 << 62), 2),
    (dict(dim=0), 2), (dict(dim=16), 2), (dict(dim=48), 2), (dict(dim=288), 2), (dict(dim=-32), 2),
    (dict(rows=256, n_pos=(1 << 31) - 1), 2),
]
FLOATS = [
    (dict(T=0), 2), (dict(T=-1), 2), (dict(T=1 << 31), 2),
    (dict(ld_tok=60), 2), (dict(ld_row=60), 2), (dict(ld_tok=-64), 2), (dict(ld_row=-640), 2),
    (dict(ld_tok=1 << 62), 2), (dict(ld_row=1 << 62), 2), (dict(ld_tok=66), 3), (dict(ld_row=642), 3),
    (dict(kc=off(KC, 8)), 3), (dict(kw=off(KW, 4)), 3), (dict(vc=off(VC, 1)), 3), (dict(vw=off(VW, 2)), 3),
    (dict(k=off(K, 4)), 3), (dict(v=off(V, 8)), 3), (dict(pos=off(POS, 4)), 3), (dict(lens=off(LENS, 4)), 3),
]
MISSING = [(dict([(n, None)]), 1) for n in ("k", "v", "kc", "kw", "vc", "vw")]


@pytest.mark.parametrize("over,status", SIZES + FLOATS + MISSING + [
    (dict(pos=None), 1), (dict(src=3), 4), (dict(src=-1), 4), (dict(src=1, ld_tok=68), 3),
    (dict(kc=K), 1), (dict(kw=off(K, 64)), 1), (dict(vc=off(V, 1024)), 1), (dict(vw=POS), 1), (dict(kc=LENS), 1),
    (dict(vc=KC), 1), (dict(vw=KC), 1), (dict(kw=off(KC, 2 * 2 * 64 * 16 - 16)), 1), (dict(vw=KW), 1)])
def test_kvq_store_refuses(lib, over, status):
    assert store(lib, **over) == status


@pytest.mark.parametrize("over,status", SIZES + FLOATS + MISSING + [
    (dict(dst=3), 4), (dict(dst=1, ld_tok=68), 3),
    (dict(k=KC), 1), (dict(v=off(KW, 16)), 1), (dict(k=POS), 1), (dict(v=LENS), 1), (dict(v=K), 1),
    (dict(v=off(K, 128)), 1),                                  # columns that overlap
    (dict(v=off(K, 256)), 1),                                  # K's next token
    (dict(ld_row=320), 2), (dict(ld_row=576), 2), (dict(ld_tok=96, ld_row=64), 2),     # rows into one another
    (dict(v=off(K, 256), ld_tok=112, ld_row=1120), 1), (dict(v=off(K, 256), ld_tok=128, ld_row=1264), 1)])
def test_kvq_load_refuses(lib, over, status):
    assert load(lib, **over) == status


def attn(lib, **over):
    a = dict(q=Q, ldq=256, kind=1, kc=KC, kw=KW, vc=VC, vw=VW, rows=2, n_pos=64, heads=8, kv_heads=2, dim=32, pos=POS,
             window=-1, sinks=0, scale=0.1, out=OUT, ldo=256, acc=None, ws=WS, wsb=0, stream=None)
    a.update(over)
    return lib.kvq_attn_decode(*a.values())


@pytest.mark.parametrize("over,status", SIZES + [
    (dict([(n, None)]), 1) for n in ("q", "kc", "kw", "vc", "vw", "pos", "out")] + [
    (dict(heads=7), 2), (dict(heads=0), 2), (dict(heads=1), 2), (dict(heads=1026, ldq=1 << 20), 2),
    (dict(heads=1 << 62), 2), (dict(window=-2), 2), (dict(sinks=-1), 2),
    (dict(ldq=255), 2), (dict(ldo=255), 2), (dict(ldq=-256), 2), (dict(ldq=1 << 62), 2),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=1e-40), 1), (dict(scale=3e38), 1),
    (dict(scale=0.0), 7),
    (dict(q=off(Q, 4)), 3), (dict(kc=off(KC, 8)), 3), (dict(kw=off(KW, 8)), 3), (dict(vc=off(VC, 4)), 3),
    (dict(vw=off(VW, 4)), 3), (dict(pos=off(POS, 4)), 3), (dict(out=off(OUT, 4)), 3), (dict(acc=off(ACC, 4)), 3),
    (dict(out=Q), 1), (dict(out=off(Q, 1024)), 1), (dict(out=off(KC, 64)), 1), (dict(out=KW), 1), (dict(out=VC), 1),
    (dict(out=off(VW, 16)), 1), (dict(out=POS), 1), (dict(acc=OUT), 1), (dict(acc=off(KC, 16)), 1), (dict(acc=VW), 1),
    (dict(acc=Q), 1), (dict(acc=POS), 1),
    (dict(ws=None), 7), (dict(wsb=16), 7), (dict(ws=off(WS, 8), wsb=BIG), 3),
    (dict(ws=KC, wsb=BIG), 1), (dict(ws=VW, wsb=BIG), 1), (dict(ws=Q, wsb=BIG), 1), (dict(ws=POS, wsb=BIG), 1),
    (dict(ws=off(OUT, -4096), wsb=BIG), 1), (dict(ws=ACC, acc=ACC, wsb=BIG), 1)])
def test_kvq_attn_decode_refuses(lib, over, status):
    assert attn(lib, **over) == status


def test_kvq_attn_decode_workspace_sizes(lib):
    f = lib.kvq_attn_decode_workspace
    plain, with_acc = f(2, 8, 2, 32, 64, -1, 0, 0), f(2, 8, 2, 32, 64, -1, 0, 1)
    assert 0 < plain <= with_acc
    assert attn(lib, wsb=plain - 1) == 7 and attn(lib, acc=ACC, wsb=with_acc - 1) == 7
    assert f(1, 8, 2, 32, 1 << 20, 128, 4, 1) < f(1, 8, 2, 32, 1 << 20, -1, 0, 1)
    for bad in ((0, 8, 2, 32, 64, -1, 0, 0), (2, 7, 2, 32, 64, -1, 0, 0), (2, 8, 2, 40, 64, -1, 0, 0),
                (2, 8, 2, 32, 0, -1, 0, 0), (2, 8, 2, 32, 64, -5, 0, 0), (2, 8, 2, 32, 64, -1, -1, 0)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kind", [0, 1])
def test_kvq_attn_decode_workspace_knows_the_largest_cache(lib, kind):
    far = dict(kind=kind, rows=256, wsb=0, **{n: C.c_void_p((i + 1) << 45) for i, n in
                                              enumerate(("q", "kc", "kw", "vc", "vw", "pos", "out", "ws"))})
    most = 1 << 25                                             # 2^39 values
    for n_pos, status in ((most, 7), (most + 1, 2)):
        assert attn(lib, n_pos=n_pos, **far) == status
        assert (lib.kvq_attn_decode_workspace(256, 8, 2, 32, n_pos, 64, 0, 0) == 0) == (status == 2)


def evict(lib, **over):
    a = dict(kind=1, kc=KC, kw=KW, vc=VC, vw=VW, rows=2, n_pos=64, kv_heads=2, dim=32, pos=POS, acc=ACC, budget=32,
             sinks=2, recent=4, new_pos=NPOS, new_acc=NACC, kept=KEPT, ws=WS, wsb=0, stream=None)
    a.update(over)
    return lib.kvq_evict(*a.values())


@pytest.mark.parametrize("over,status", SIZES + [
    (dict([(n, None)]), 1) for n in ("kc", "kw", "vc", "vw", "pos", "acc", "new_pos", "new_acc")] + [
    (dict(budget=0), 2), (dict(budget=65), 2), (dict(sinks=-1), 2), (dict(recent=-1), 2), (dict(sinks=33), 2),
    (dict(sinks=20, recent=13), 2), (dict(sinks=1, recent=(1 << 63) - 1), 2),
    (dict(kc=off(KC, 8)), 3), (dict(kw=off(KW, 4)), 3), (dict(vc=off(VC, 8)), 3), (dict(vw=off(VW, 4)), 3),
    (dict(pos=off(POS, 4)), 3), (dict(acc=off(ACC, 4)), 3), (dict(new_pos=off(NPOS, 4)), 3),
    (dict(new_acc=off(NACC, 4)), 3), (dict(kept=off(KEPT, 4)), 3),
    (dict(ws=None), 7), (dict(wsb=16), 7), (dict(ws=off(WS, 4), wsb=BIG), 3)])
def test_kvq_evict_refuses(lib, over, status):
    assert evict(lib, **over) == status


@pytest.mark.parametrize("over", [
    dict(vc=off(KC, 256)), dict(kw=KC), dict(vw=off(VC, 4096 - 16)), dict(new_acc=off(ACC, 16)),
    dict(new_pos=off(POS, -16), rows=8), dict(new_acc=KC), dict(kept=VC), dict(kept=ACC), dict(kept=NACC),
    dict(new_pos=KEPT), dict(pos=KW), dict(acc=VW), dict(ws=KC), dict(ws=NACC), dict(ws=off(KEPT, -4096)),
    dict(ws=POS), dict(ws=ACC), dict(ws=NPOS)])
def test_kvq_evict_refuses_buffers_that_overlap(lib, over):
    assert evict(lib, wsb=BIG, **over) == 1


def test_kvq_evict_workspace_sizes(lib):
    f = lib.kvq_evict_workspace
    assert f(2, 2, 32) == lib.kv_evict_workspace(2, 2, 32) > 0
    assert evict(lib, wsb=f(2, 2, 32) - 1) == 7
    assert evict(lib, new_pos=POS, new_acc=ACC, wsb=f(2, 2, 32) - 1) == 7   # in place: allowed so far
    assert f(0, 2, 32) == 0 and f(2, 0, 32) == 0 and f(2, 2, 0) == 0


@pytest.mark.parametrize("source", ["kvq.cu", "kvq.cuh", "attn_kvq.cuh"])
def test_no_read_only_loads(source):
    """These grids begin while the one before may still write what they read."""
    with open(os.path.join(build.CSRC, source)) as f:
        text = f.read()
    assert "__ldg(" not in text and ".nc" not in text


def test_binding_refuses_host_tensors_and_odd_heads():
    pytest.importorskip("torch")
    cache = native.kvq_cache("u4", 1, 8, 1, 32, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(1, 1, 8, 16), (1, 1, 8, 1, 2)] * 2
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        native.kvq_store(cache[0], cache[0], cache[0], cache)
    for dim in (0, 16, 40, 288):
        with pytest.raises(ValueError):
            native.kvq_cache("i8", 1, 8, 1, dim, device="cpu")


# kvq_load's buffers, by enumeration.  Accepted calls have placeholder pointers, so they run in a process
# that sees no GPU: it ends them with Q8_ERR_CUDA before any launch.
_PLACES = r"""
import ctypes as C, random, sys
from q8_quantized_projection_gb300 import native
lib = native.load()
assert lib.q8_last_cuda_error() == 0
W = 32                                        # values of a run: one head of 32, in f32 or 16 bits

def load(k, v, pos, lens, planes, rows, T, ld_row, ld_tok, dst, n_pos, kind=1):
    P = lambda x: C.c_void_p(x) if x else None
    return lib.kvq_load(kind, *map(P, planes), rows, n_pos, 1, W, P(pos), T, P(lens), dst, P(k), P(v), ld_row, ld_tok, None)

def runs(p, rows, T, ld_row, ld_tok, elt):
    return [(p + (m * ld_row + t * ld_tok) * elt, p + (m * ld_row + t * ld_tok + W) * elt)
            for m in range(rows) for t in range(T)]

def meet(a, b):
    return any(x < w and u < y for x, y in a for u, w in b)

M = 1 << 20
far = [100 * M, 104 * M, 108 * M, 112 * M]
OPEN = 5
assert load(M, 2 * M, 3 * M, 0, far, 2, 3, 96, 32, 0, 16) == OPEN
# one token of one row, whatever lies between its K and its V, and whatever its strides say
for ld_row, ld_tok in ((32, 32), (0, 0), (-7, 1), (1 << 62, -1 << 62)):
    for dst in (0, 1, 2):
        assert load(M, 9 * M, 6 * M, 7 * M, far, 1, 1, ld_row, ld_tok, dst, 16) == OPEN
        assert load(200 * M, M, 50 * M, 60 * M, far, 1, 1, ld_row, ld_tok, dst, 16) == OPEN
# K and V as halves of [rows][2][T][W]
assert load(M, M + 4 * W * 4, 2 * M, 0, far, 3, 4, 8 * W, W, 0, 16) == OPEN
# one token a row, a pitch longer than from K to V
assert load(M, 9 * M, 6 * M, 0, far, 2, 1, 4 * M, 0, 0, 16) == OPEN
rng = random.Random(1)
seen = {1: 0, OPEN: 0}
for i in range(20000):
    dst, rows, T = rng.choice((0, 1, 2)), rng.choice((1, 1, 2, 3, 5)), rng.choice((1, 1, 2, 3, 4))
    elt = 2 if dst else 4
    step = 16 // elt
    if rng.random() < 0.5:
        ld_tok = W + step * rng.choice((0, 0, 1, 4, rng.randrange(40)))
        ld_row = (T - 1) * ld_tok + W + step * rng.choice((0, 0, 3, rng.randrange(60)))
    else:
        ld_row = W + step * rng.choice((0, 0, 1, 4, rng.randrange(40)))
        ld_tok = (rows - 1) * ld_row + W + step * rng.choice((0, 0, 3, rng.randrange(60)))
    if rows == 1: ld_row = rng.choice((ld_row, 0, 3))
    if T == 1: ld_tok = rng.choice((ld_tok, 0, 3))
    span = 16 * rng.choice((8, 64, 160, 400))
    n_pos = rng.choice((1, 2, 5))
    at = lambda: M + 16 * rng.randrange(span // 16) if rng.random() < 0.4 else M * rng.randrange(2, 90)
    k, v = M, M + 16 * rng.randrange(-span // 16, span // 16)
    pos, lens, planes = at(), at() if rng.random() < 0.5 else 0, [at() for _ in range(4)]
    both = runs(k, rows, T, ld_row, ld_tok, elt), runs(v, rows, T, ld_row, ld_tok, elt)
    others = [(pos, pos + 4 * rows)] + [(lens, lens + 4 * rows)] * (lens > 0)
    others += [(p, p + rows * n_pos * (W // 2, 4)[j % 2]) for j, p in enumerate(planes)]
    want = 1 if meet(*both) or meet(both[0] + both[1], others) else OPEN
    got = load(k, v, pos, lens, planes, rows, T, ld_row, ld_tok, dst, n_pos)
    assert got == want, (i, got, want, dst, rows, T, ld_row, ld_tok, v - k, pos - k, lens and lens - k, [p - k for p in planes], n_pos)
    seen[got] += 1
assert min(seen.values()) > 2000, seen
print("checked", seen)
"""


def test_kvq_load_refuses_what_overlaps_and_nothing_else(lib):
    """Among strided runs of K and V, whatever lies between them untouched."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=build.ROOT)
    r = subprocess.run([sys.executable, "-c", _PLACES], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "checked" in r.stdout, r.stdout + r.stderr
