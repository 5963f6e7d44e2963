"""GPU tests of attn_decode's precision: inputs whose result hangs on low bits, on small
weights or on every part of a long row (attn_precision.py has them and their bounds)."""
import numpy as np
import pytest

import attn_precision as ap
from q8_quantized_projection_gb300 import native

pytestmark = pytest.mark.gpu
KVS, DIMS = ["f32", "f16", "bf16"], [64, 80, 128, 200, 256]


def run(kv, q, k, v, scale=ap.SCALE):
    """attn_decode of q [rows][heads][D] on one K/V head's k, v [rows][n][D]: out, weights."""
    import torch as t
    rows, heads, dim = q.shape
    n = k.shape[1]
    ty = {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[kv]
    dev = lambda x, ty: t.from_numpy(np.ascontiguousarray(x)).to("cuda").to(ty)  # noqa: E731
    out, acc = t.empty(rows, heads * dim, device="cuda"), t.zeros(rows, 1, n, device="cuda")
    kd, vd = dev(k, ty), dev(v, ty)
    assert np.array_equal(vd.double().cpu().numpy(), v)
    native.attn_decode(dev(q.reshape(rows, -1), t.float32), kd, vd, t.full((rows,), n - 1, dtype=t.int32, device="cuda"),
                       out, native.attn_workspace(rows, heads, 1, dim, n, acc=True), heads, 1, scale=scale, acc=acc)
    assert native.q8_device_error() == 0
    return out.double().cpu().numpy().reshape(rows, heads, dim), acc.double().cpu().numpy()[:, 0], kd.double().cpu().numpy()


def check(got, want, tol):
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("heads", [2, 4, 5, 8])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("n,at", [(16, 0), (300, 5)])
def test_small_weights_beside_large_ones_of_no_value(kv, heads, dim, n, at):
    q, k, v = ap.small_weights(heads, dim, n, at)
    want, p = ap.exact(q, k, v)
    got, acc, _ = run(kv, q, k, v)
    check(got, want, ap.small_weights_bound(want, n))
    # (acc: the heads' sum, one rounding a head and one into acc)
    check(acc, p.sum(1), ap.small_weights_bound(p.sum(1), n) + (heads + 1) * ap.U * p.sum(1))


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("heads", [4, 8])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("n", [64, 600])
def test_weights_that_cancel(kv, heads, dim, n):
    q, k, v = ap.cancelling_weights(heads, dim, n)
    want, _ = ap.exact(q, k, v)
    check(run(kv, q, k, v)[0], want, ap.cancelling_weights_bound(want, n))


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("heads", [4, 7, 8])
@pytest.mark.parametrize("dim", DIMS)
def test_low_parts_of_q(kv, heads, dim):
    q, k, v = ap.low_parts_of_q(kv, heads, dim)
    want, p = ap.exact(q, k, v)
    got, acc, kd = run(kv, q, k, v)
    assert np.array_equal(kd, k)
    check(got, want, ap.low_parts_of_q_bound(want, kv, heads, dim))
    check(acc, p.sum(1), ap.low_parts_of_q_bound(p.sum(1), kv, heads, dim) + (heads + 1) * ap.U * p.sum(1))


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("heads", [4, 7, 8])
@pytest.mark.parametrize("dim", DIMS)
def test_small_values_of_q_beside_a_large_one(kv, heads, dim):
    q, k, v = ap.small_values_of_q(heads, dim)
    want, _ = ap.exact(q, k, v)
    check(run(kv, q, k, v)[0], want, ap.small_values_of_q_bound(want, dim))


@pytest.mark.parametrize("kv,heads,dim,n", [
    ("f32", 8, 256, 9000), ("f32", 8, 72, 20000), ("f32", 5, 8, 30000), ("f32", 1, 64, 60000), ("f32", 1, 8, 70000),
    ("f32", 2, 200, 20000), ("bf16", 8, 128, 30000), ("bf16", 3, 24, 60000), ("bf16", 1, 256, 40000),
    ("f16", 7, 40, 30000), ("f16", 4, 200, 20000), ("f16", 6, 256, 15000)])
def test_every_part_of_a_long_row_counts(kv, heads, dim, n):
    """V is 1 in one slice of the row a column, so that a part lost or misweighed in the join moves a column."""
    r = np.random.default_rng(n + dim)
    q = r.standard_normal((1, heads, dim)).astype(np.float32).astype(np.float64)
    to = {"f32": lambda x: x.astype(np.float32).astype(np.float64), "f16": ap.to_f16, "bf16": ap.to_bf16}[kv]
    k, v = to(r.standard_normal((1, n, dim))), ap.sliced_values(n, dim)[None]
    scale = dim ** -0.5
    want, p = ap.exact(q * scale / np.log(2), k, v)
    got, acc, kd = run(kv, q, k, v, scale)
    assert np.array_equal(kd, k)
    check(got[0], want[0], ap.long_row_bound(q[0], k[0], want[0], scale))
    check(acc[0], p[0].sum(0), ap.long_row_bound(q[0], k[0], p[0], scale).sum(0) + (heads + 1) * ap.U * p[0].sum(0))
