"""Pins of the oracles of the row operators and the block norms: invariants of the permutation, and
every gradient against central differences of the forward computation (float64)."""
import numpy as np
import pytest

from oracle import block_norm as bn
from oracle import rows as ro


def _difference(f, v, out_grad, eps=1e-6):
    """d <f(v), out_grad> / dv by central differences, one element at a time."""
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        up, dn = v.copy(), v.copy()
        up[i] += eps
        dn[i] -= eps
        g[i] = (np.sum(f(up) * out_grad) - np.sum(f(dn) * out_grad)) / (2 * eps)
    return g


@pytest.mark.parametrize("capacity", [0, 1, 3])
def test_permutation_with_dropped_pairs(capacity):
    rng = np.random.default_rng(capacity)
    E = 5
    ids = rng.integers(-2, E + 2, 40)
    off, pair, row, lst = ro.permute_capacity(ids, E, capacity)
    assert sorted(pair) == list(range(40))
    for e in range(E):
        held = pair[off[e]:off[e + 1]]
        assert list(held) == sorted(held) and all(ids[p] == e for p in held)
        n = int((ids == e).sum())
        assert len(held) == (n if capacity == 0 else min(n, capacity))
        assert all(row[p] == off[e] + i for i, p in enumerate(held))
    tail = pair[off[E]:]
    assert list(tail) == sorted(tail) and all(row[p] == -1 for p in tail)
    assert list(lst[1:1 + lst[0]]) == [e for e in range(E) if off[e + 1] > off[e]]


def test_row_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, k, H, E = 3, 2, 4, 3
    ids = np.array([0, 2, 1, -1, 2, 2])
    _, _, row, _ = ro.permute_capacity(ids, E, 2)
    x, w = rng.standard_normal((T, H)), rng.standard_normal(T * k)
    rows, zero = rng.standard_normal((T * k, H)), np.zeros((T * k, H))
    used = np.zeros((T * k, 1))
    used[row[row >= 0]] = 1.0
    d_rows = rng.standard_normal((T * k, H)) * used
    dx = _difference(lambda v: ro.sort_rows(v, w, row, k, zero), x, d_rows)
    dw = _difference(lambda v: ro.sort_rows(x, v, row, k, zero), w, d_rows)
    assert np.allclose(dx, ro.unsort_rows(d_rows, w, row, T, k), atol=1e-8)
    assert np.allclose(dw, ro.pair_dots(d_rows, x, row, k), atol=1e-8)
    d_out = rng.standard_normal((T, H))
    dr = _difference(lambda v: ro.unsort_rows(v, w, row, T, k), rows, d_out)
    dw = _difference(lambda v: ro.unsort_rows(rows, v, row, T, k), w, d_out)
    assert np.allclose(dr, ro.sort_rows(d_out, w, row, k, zero), atol=1e-8)
    assert np.allclose(dw, ro.pair_dots(rows, d_out, row, k), atol=1e-8)


def test_router_softmax_gradient_against_differences():
    rng = np.random.default_rng(1)
    T, E, k = 3, 6, 3
    logits, dw = rng.standard_normal((T, E)), rng.standard_normal(T * k)
    ids = np.argsort(-logits, axis=1)[:, :k]

    def weights(l):
        v = np.take_along_axis(l, ids, 1)
        e = np.exp(v - v.max(1, keepdims=True))
        return (e / e.sum(1, keepdims=True)).reshape(-1)

    ref = _difference(weights, logits, dw)
    assert np.allclose(ref, ro.route_topk_bwd(dw, weights(logits), ids.reshape(-1), T, E, k), atol=1e-8)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "token", "full"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_block_norm_gradient_against_differences(post, gate, sigmoid):
    rng = np.random.default_rng(2)
    T, H = 3, 5
    r = rng.standard_normal
    x, y, dz, dh = r((T, H)), r((T, H)), r((T, H)), r((T, H))
    wp, wn = (r(H) if post else None), r(H)
    g = {None: None, "token": r(T), "full": r((T, H))}[gate]
    kw = dict(sigmoid=sigmoid, alpha=0.7, eps=1e-3)

    def total(x=x, y=y, wp=wp, g=g, wn=wn):
        z, h = bn.block_norm(x, y, wp, g, w_next=wn, **kw)
        return np.stack([z, h])

    dout = np.stack([dz, dh])
    z, _ = bn.block_norm(x, y, wp, g, w_next=wn, **kw)
    got = bn.block_norm_bwd(z, dz, dh, y, wp, g, w_next=wn, **kw)
    assert np.allclose(got["dx"], _difference(lambda v: total(x=v), x, dout), atol=1e-7)
    assert np.allclose(got["dy"], _difference(lambda v: total(y=v), y, dout), atol=1e-7)
    assert np.allclose(got["dw_next"], _difference(lambda v: total(wn=v), wn, dout), atol=1e-7)
    if post:
        assert np.allclose(got["dw_post"], _difference(lambda v: total(wp=v), wp, dout), atol=1e-7)
    if gate:
        assert np.allclose(got["dgate"], _difference(lambda v: total(g=v), g, dout), atol=1e-7)
