"""Host-side checks of attn_decode, kv_evict and head_sample: what they refuse,
before anything touches a GPU, and their workspaces' sizes."""
import ctypes as C
import os

import pytest

from q8_quantized_projection_gb300 import build, native


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def P(n):
    """A 16-byte aligned placeholder pointer (never dereferenced), far from P of another n."""
    return C.c_void_p((n + 1) << 32)


Q, K, V, POS, OUT, ACC, WS, NPOS, NACC, KEPT = (P(i) for i in range(10))
BIG = 1 << 40


def off(p, n):
    return C.c_void_p(p.value + n)


def attn(lib, **over):
    a = dict(q=Q, ldq=256, k=K, v=V, kv=0, rows=2, n_pos=64, heads=8, kv_heads=2, dim=32, pos=POS,
             window=-1, sinks=0, scale=0.1, out=OUT, ldo=256, acc=None, ws=WS, wsb=0, stream=None)
    a.update(over)
    return lib.attn_decode(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1), (dict(out=None), 1),
    (dict(kv=3), 4), (dict(kv=-1), 4),
    (dict(rows=0), 2), (dict(rows=257), 2), (dict(n_pos=0), 2), (dict(n_pos=1 << 31), 2),
    (dict(heads=7), 2), (dict(heads=0), 2), (dict(heads=1), 2), (dict(heads=1026, ldq=1 << 20), 2),
    (dict(kv_heads=0), 2), (dict(kv_heads=1 << 62), 2), (dict(heads=1 << 62), 2),
    (dict(dim=0), 2), (dict(dim=12), 2), (dict(dim=264), 2), (dict(dim=-8), 2),
    (dict(rows=256, n_pos=(1 << 31) - 1), 2),                 # a cache beyond 2^40 bytes
    (dict(window=-2), 2), (dict(sinks=-1), 2),
    (dict(ldq=255), 2), (dict(ldo=255), 2), (dict(ldq=-256), 2), (dict(ldq=1 << 62), 2),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q=off(Q, 4)), 3), (dict(k=off(K, 8)), 3), (dict(v=off(V, 4)), 3), (dict(pos=off(POS, 4)), 3),
    (dict(out=off(OUT, 4)), 3), (dict(acc=off(ACC, 4)), 3),
    (dict(out=Q), 1), (dict(out=off(Q, 1024)), 1), (dict(out=off(K, 64)), 1), (dict(out=V), 1),
    (dict(out=POS), 1), (dict(acc=OUT), 1), (dict(acc=off(K, 16)), 1), (dict(acc=Q), 1), (dict(acc=POS), 1),
    (dict(ws=None), 7), (dict(wsb=16), 7), (dict(ws=off(WS, 8), wsb=BIG), 3),
    (dict(ws=K, wsb=BIG), 1), (dict(ws=Q, wsb=BIG), 1), (dict(ws=off(OUT, -4096), wsb=BIG), 1),
    (dict(ws=POS, wsb=BIG), 1), (dict(ws=ACC, acc=ACC, wsb=BIG), 1),
])
def test_attn_decode_refuses(lib, over, status):
    assert attn(lib, **over) == status


@pytest.mark.parametrize("scale,status", [
    (3e38, 1), (-3.4e38, 1), (1.8e38, 1), (1e-38, 1), (-1e-45, 1),
    (0.0, 7), (-0.0, 7), (2.0 ** 127, 7), (-2.0 ** 127, 7), (2.0 ** -126, 7), (-2.0 ** -126, 7)])
def test_attn_decode_scale(lib, scale, status):
    """Refused where its product with log2(e) would overflow (0 times infinity is NaN) or lose bits."""
    assert attn(lib, scale=scale) == status


def test_attn_decode_workspace_sizes(lib):
    f = lib.attn_decode_workspace
    plain, with_acc = f(2, 8, 2, 32, 64, -1, 0, 0), f(2, 8, 2, 32, 64, -1, 0, 1)
    assert 0 < plain <= with_acc
    assert attn(lib, wsb=plain - 1) == 7
    assert attn(lib, acc=ACC, wsb=with_acc - 1) == 7
    # a window bounds what is kept of the scores, however long the cache
    assert f(1, 8, 2, 32, 1 << 20, 128, 4, 1) < f(1, 8, 2, 32, 1 << 20, -1, 0, 1)
    assert f(1, 8, 2, 32, 64, (1 << 63) - 1, (1 << 63) - 1, 1) == f(1, 8, 2, 32, 64, -1, 0, 1)
    for bad in ((0, 8, 2, 32, 64, -1, 0, 0), (2, 7, 2, 32, 64, -1, 0, 0), (2, 8, 2, 20, 64, -1, 0, 0),
                (2, 8, 2, 32, 0, -1, 0, 0), (2, 8, 2, 32, 64, -5, 0, 0), (2, 8, 2, 32, 64, -1, -1, 0)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kv", [0, 1, 2])
def test_attn_decode_workspace_knows_the_largest_cache(lib, kv):
    """The workspace's size has no cache type: it is 0 exactly where the call refuses the sizes."""
    far = dict(kv=kv, rows=256, wsb=0, **{n: C.c_void_p((i + 1) << 45) for i, n in
                                          enumerate(("q", "k", "v", "pos", "out", "ws"))})
    most = 1 << 25                                             # 2^39 values
    for n_pos, status in ((most // 2 + 1, 7), (most, 7), (most + 1, 2)):
        assert attn(lib, n_pos=n_pos, **far) == status
        assert (lib.attn_decode_workspace(256, 8, 2, 32, n_pos, 64, 0, 0) == 0) == (status == 2)


def evict(lib, **over):
    a = dict(k=K, v=V, kv=0, rows=2, n_pos=64, kv_heads=2, dim=32, pos=POS, acc=ACC, budget=32, sinks=2,
             recent=4, new_pos=NPOS, new_acc=NACC, kept=KEPT, ws=WS, wsb=0, stream=None)
    a.update(over)
    return lib.kv_evict(*a.values())


OVERLAPS = [
    dict(v=off(K, 256)), dict(new_acc=off(ACC, 16)), dict(new_pos=off(POS, -16), rows=8), dict(new_acc=K),
    dict(kept=V), dict(kept=ACC), dict(kept=NACC), dict(new_pos=KEPT), dict(pos=K), dict(acc=V),
    dict(ws=K), dict(ws=NACC), dict(ws=off(KEPT, -4096)), dict(ws=POS), dict(ws=ACC), dict(ws=NPOS)]


@pytest.mark.parametrize("over", OVERLAPS)
def test_kv_evict_refuses_buffers_that_overlap(lib, over):
    assert evict(lib, wsb=BIG, **over) == 1


@pytest.mark.parametrize("over,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1), (dict(acc=None), 1), (dict(new_pos=None), 1),
    (dict(new_acc=None), 1), (dict(kv=3), 4), (dict(rows=0), 2), (dict(rows=257), 2), (dict(n_pos=0), 2),
    (dict(dim=4), 2), (dict(kv_heads=0), 2), (dict(kv_heads=1025), 2),
    (dict(budget=0), 2), (dict(budget=65), 2), (dict(sinks=-1), 2), (dict(recent=-1), 2),
    (dict(sinks=33), 2), (dict(sinks=20, recent=13), 2), (dict(sinks=1, recent=(1 << 63) - 1), 2),
    (dict(k=off(K, 8)), 3), (dict(v=off(V, 8)), 3), (dict(pos=off(POS, 4)), 3), (dict(acc=off(ACC, 4)), 3),
    (dict(new_pos=off(NPOS, 4)), 3), (dict(new_acc=off(NACC, 4)), 3), (dict(kept=off(KEPT, 4)), 3),
    (dict(ws=None), 7), (dict(wsb=16), 7), (dict(ws=off(WS, 4), wsb=BIG), 3),
])
def test_kv_evict_refuses(lib, over, status):
    assert evict(lib, **over) == status


def test_kv_evict_workspace_sizes(lib):
    f = lib.kv_evict_workspace
    assert f(2, 2, 32) >= 2 * 2 * 32 * 4
    assert evict(lib, wsb=f(2, 2, 32) - 1) == 7
    assert evict(lib, new_pos=POS, new_acc=ACC, wsb=f(2, 2, 32) - 1) == 7   # in place: allowed so far
    assert f(0, 2, 32) == 0 and f(2, 0, 32) == 0 and f(2, 2, 0) == 0 and f(2, 2, 1 << 31) == 0


def sample(lib, **over):
    a = dict(x=Q, ldl=100, rows=2, n=100, u=P(11), t=P(12), k=P(13), p=P(14), mp=P(15), tok=P(16), prob=P(17),
             kept=P(18), stream=None)
    a.update(over)
    return lib.head_sample(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(x=None), 1), (dict(u=None), 1), (dict(tok=None), 1),
    (dict(rows=0), 2), (dict(rows=257), 2), (dict(n=0), 2), (dict(n=(1 << 20) + 1, ldl=1 << 21), 2),
    (dict(ldl=99), 2), (dict(ldl=1 << 62), 2),
    (dict(x=off(Q, 4)), 3), (dict(u=off(P(11), 2)), 3), (dict(t=off(P(11), 1)), 3), (dict(k=off(P(11), 2)), 3),
    (dict(p=off(P(11), 2)), 3), (dict(mp=off(P(11), 2)), 3), (dict(tok=off(P(11), 2)), 3),
    (dict(prob=off(P(11), 2)), 3), (dict(kept=off(P(11), 2)), 3),
])
def test_head_sample_refuses(lib, over, status):
    assert sample(lib, **over) == status


@pytest.mark.parametrize("over", [
    dict(prob=P(12)), dict(prob=off(P(12), 4)), dict(prob=off(P(11), -4)), dict(prob=P(14)), dict(prob=P(15)),
    dict(tok=P(13)), dict(tok=P(12)), dict(tok=P(11)), dict(kept=P(13)), dict(kept=P(12)),
    dict(prob=P(16)), dict(kept=P(16)), dict(kept=off(P(17), 4)),
    dict(tok=Q), dict(prob=off(Q, 4 * 199)), dict(kept=off(Q, 400)), dict(prob=off(Q, -4)),
    dict(tok=P(13), prob=None, kept=None), dict(ldl=1 << 20, tok=off(Q, 4 << 20))])
def test_head_sample_refuses_outputs_that_overlap(lib, over):
    """In place: one CTA of a row could read settings that another has written over."""
    assert sample(lib, **over) == 1


@pytest.mark.parametrize("source", ["attn.cu", "attn.cuh", "attn_mma.cuh", "evict.cu", "sample.cu"])
def test_no_read_only_loads(source):
    """These grids begin while the one before may still write what they read (they wait for it on
    the device), so nothing may go through the path for memory that is read-only while a grid runs."""
    with open(os.path.join(build.CSRC, source)) as f:
        text = f.read()
    assert "__ldg(" not in text and ".nc" not in text


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 8)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        native.head_sample(x, torch.zeros(1), torch.zeros(1, dtype=torch.int32))
