"""The fp64 oracles of layer norm, rotary positions and attention, on the CPU:
their gradients against central differences, and properties that follow from
the definitions alone.

Differences: the losses are smooth with derivatives of order one, so a step of
1e-5 leaves a truncation error of about 1e-10 and a rounding error of about
1e-16 / 1e-5 * |loss| ~ 1e-10; the bar is 1e-7 of the largest gradient entry.
"""
import numpy as np
import pytest

from oracle import ops

H = 1e-5


def differences(loss, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += H
        dn[i] -= H
        g[i] = (loss(up) - loss(dn)) / (2 * H)
    return g


def close(got, ref, name):
    bar = 1e-7 * max(1.0, np.abs(ref).max())
    assert np.abs(got - ref).max() <= bar, (name, np.abs(got - ref).max(), bar)


def test_layer_norm_gradients():
    r = np.random.default_rng(0)
    x, w, b, dy = r.standard_normal((3, 7)), r.standard_normal(7), r.standard_normal(7), r.standard_normal((3, 7))
    dx, dw, db = ops.layer_norm_bwd(dy, x, w)
    close(differences(lambda t: (ops.layer_norm(t, w, b)[0] * dy).sum(), x), dx, "dx")
    close(differences(lambda t: (ops.layer_norm(x, t, b)[0] * dy).sum(), w), dw, "dw")
    close(differences(lambda t: (ops.layer_norm(x, w, t)[0] * dy).sum(), b), db, "db")


@pytest.mark.parametrize("halves", [False, True])
def test_rotary_is_an_inverse_and_a_gradient(halves):
    r = np.random.default_rng(1)
    x, dy = r.standard_normal((5, 2, 12)), r.standard_normal((5, 2, 12))
    pos = r.integers(0, 1000, (5, 3))
    axes = (4, 2, 4)
    y = ops.rotary(x, pos, axes, halves=halves)
    np.testing.assert_allclose(ops.rotary(y, pos, axes, halves=halves, inverse=True), x, atol=1e-13)
    np.testing.assert_array_equal(y[..., 10:], x[..., 10:])
    dx = ops.rotary(dy, pos, axes, halves=halves, inverse=True)
    close(differences(lambda t: (ops.rotary(t, pos, axes, halves=halves) * dy).sum(), x), dx, "dx")
    # products of queries and keys depend on the distance alone
    k = r.standard_normal((5, 2, 12))
    a = (ops.rotary(x, pos, axes, halves=halves) * ops.rotary(k, pos + 3, axes, halves=halves)).sum(-1)
    b = (ops.rotary(x, pos + 9, axes, halves=halves) * ops.rotary(k, pos + 12, axes, halves=halves)).sum(-1)
    np.testing.assert_allclose(a, b, atol=1e-11)


@pytest.mark.parametrize("lq,lk,causal,block", [(4, 6, False, 1), (5, 5, True, 1), (6, 4, True, 1), (5, 7, True, 3)])
def test_attention_gradients(lq, lk, causal, block):
    r = np.random.default_rng(2)
    q, do = r.standard_normal((2, lq, 4, 3))
    k, v = r.standard_normal((2, lk, 2, 3))
    kw = dict(causal=causal, block=block)
    dq, dk, dv = ops.attention_bwd(q, k, v, do, **kw)
    close(differences(lambda t: (ops.attention(t, k, v, **kw)[0] * do).sum(), q), dq, "dq")
    close(differences(lambda t: (ops.attention(q, t, v, **kw)[0] * do).sum(), k), dk, "dk")
    close(differences(lambda t: (ops.attention(q, k, t, **kw)[0] * do).sum(), v), dv, "dv")


def test_visible_keys():
    np.testing.assert_array_equal(ops.visible(3, 3, True), [1, 2, 3])
    np.testing.assert_array_equal(ops.visible(2, 5, True), [4, 5])
    np.testing.assert_array_equal(ops.visible(4, 2, True), [0, 0, 1, 2])          # rows that see nothing
    np.testing.assert_array_equal(ops.visible(5, 5, True, 2), [2, 2, 4, 4, 5])     # blocks of two; the last is short
    np.testing.assert_array_equal(ops.visible(2, 6, True, 4), [6, 6])
    np.testing.assert_array_equal(ops.visible(2, 0, False), [0, 0])
    o, lse = ops.attention(np.ones((4, 1, 2)), np.ones((2, 1, 2)), np.ones((2, 1, 2)), causal=True)
    np.testing.assert_array_equal(o[:2], 0)
    assert np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
