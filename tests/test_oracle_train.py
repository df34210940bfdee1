"""Pins of the oracle's training side: the gradients of the router losses, of the top-k
weights, of the finalize and of the adapters against central differences of the losses
in float64, hand cases of the balance loss, and the top-k weights against the router front.

Tolerance of a difference with step h on float64 values of size one: h^2 times a third
derivative of size one plus 2^-52 / h, with h = 1e-5 below 1e-9; 1e-7 leaves room for the
sizes of the sums."""
import numpy as np
import pytest

from oracle import train as ot
from oracle.layer import router_topk

H = 1e-5


def _differences(f, a):
    g = np.zeros(a.shape)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + H
        up = f()
        a[i] = keep - H
        down = f()
        a[i] = keep
        g[i] = (up - down) / (2 * H)
    return g


def _router(seed, T=9, E=6, K=3):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E))
    ids = np.argsort(-logits, axis=1)[:, :K].astype(np.int64)
    ids[2] = -1                     # padding
    ids[4, 1] = E                   # an id that is no expert
    return rng, logits, ids


def test_balance_by_hand():
    """Two tokens, two experts, K = 1: even load and even probabilities give 1; all on one
    expert with probabilities (3/4, 1/4) gives 2 * 3/4 = 1.5."""
    c, n, P, b, z = ot.router_balance(np.zeros((2, 2)), [[0], [1]])
    assert c.tolist() == [[1, 1]] and n.tolist() == [2] and np.allclose(P, 1.0)
    assert np.isclose(b[0], 1.0) and np.isclose(z[0], np.log(2.0) ** 2)
    l = np.log([[3.0, 1.0], [3.0, 1.0]])
    c, n, P, b, z = ot.router_balance(l, [[0], [0]])
    assert c.tolist() == [[2, 0]] and np.isclose(b[0], 1.5) and np.isclose(z[0], np.log(4.0) ** 2)


def test_balance_skips_padding_masked_rows_and_empty_sequences():
    _, logits, ids = _router(1)
    logits[5] = -np.inf
    off = [1, 4, 4, 8]
    c, n, P, b, z = ot.router_balance(logits, ids, off)
    assert n.tolist() == [2, 0, 3] and b[1] == 0 and z[1] == 0 and not c[1].any()
    assert c.sum(axis=1).tolist() == [6, 0, 8]
    keep = [1, 3]
    c1, n1, P1, b1, z1 = ot.router_balance(logits[keep], ids[keep])
    assert np.array_equal(c[0], c1[0]) and np.isclose(b[0], b1[0]) and np.isclose(z[0], z1[0])


def test_topk_weights_match_the_router_front():
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((20, 11)).astype(np.float32)
    for renorm in (False, True):
        ids, w = router_topk(logits, 4, renorm)
        np.testing.assert_allclose(ot.topk_weights(logits, ids, renorm), w, rtol=1e-6)


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_by_differences(renorm):
    rng, logits, ids = _router(5)
    off = np.array([1, 5, 5, 8])
    counts, tokens, *_ = ot.router_balance(logits, ids, off)
    db, dz = rng.standard_normal(3), rng.standard_normal(3)
    dw = rng.standard_normal(ids.shape)

    def loss():
        """The counts are held: they have no gradient."""
        _, n, P, _, z = ot.router_balance(logits, ids, off)
        K, E = ids.shape[1], logits.shape[1]
        nn = np.maximum(n, 1)
        b = E * np.sum(counts / (nn * K)[:, None] * P / nn[:, None], axis=1)
        return np.sum(db * b) + np.sum(dz * z) + np.sum(dw * ot.topk_weights(logits, ids, renorm))

    grad, size = ot.router_backward(logits, ids, counts, tokens, db, dz, dw, renorm, off)
    np.testing.assert_allclose(grad, _differences(loss, logits), atol=1e-7)
    assert np.all(np.abs(grad) <= size * (1 + 1e-12) + 1e-300)
    assert not grad[2].any()


def test_finalize_gradient_by_differences():
    rng = np.random.default_rng(7)
    T, K, Hd, R = 4, 3, 5, 10
    row = np.full(T * K, -1)
    row[rng.permutation(T * K)[:R]] = rng.permutation(R)
    row = row.reshape(T, K)
    z, w, dout = rng.standard_normal((R, Hd)), rng.standard_normal((T, K)), rng.standard_normal((T, Hd))

    def loss():
        out = np.zeros((T, Hd))
        for t in range(T):
            for j in range(K):
                if row[t, j] >= 0:
                    out[t] += w[t, j] * z[row[t, j]]
        return np.sum(out * dout)

    d_w, d_z, _ = ot.finalize_backward(dout, z, row, w)
    np.testing.assert_allclose(d_w, _differences(loss, w), atol=1e-7)
    np.testing.assert_allclose(d_z, _differences(loss, z), atol=1e-7)


def test_adapter_gradient_by_differences():
    rng = np.random.default_rng(9)
    T, n, Hd, N, R = 7, 3, 6, 5, 2
    ids = np.array([0, 2, -1, 2, 0, 3, 2])             # adapter 1 unused, 3 is none
    x, down, up = rng.standard_normal((T, Hd)), rng.standard_normal((n, R, Hd)), rng.standard_normal((n, N, R))
    scale, base, dy = rng.standard_normal(n), rng.standard_normal((T, N)), rng.standard_normal((T, N))

    def loss():
        return np.sum(ot.adapter_forward(x, ids, down, up, scale, base)[0] * dy)

    out, v = ot.adapter_forward(x, ids, down, up, scale, base)
    for t in range(T):                                 # token by token
        a = ids[t]
        want = base[t] + (scale[a] * up[a] @ (down[a] @ x[t]) if 0 <= a < n else 0.0)
        np.testing.assert_allclose(out[t], want, rtol=1e-12)
    dx, d_down, d_up, _ = ot.adapter_backward(dy, x, v, ids, down, up, scale)
    np.testing.assert_allclose(dx, _differences(loss, x), atol=1e-7)
    np.testing.assert_allclose(d_down, _differences(loss, down), atol=1e-7)
    np.testing.assert_allclose(d_up, _differences(loss, up), atol=1e-7)
    assert not d_down[1].any() and not d_up[1].any() and not dx[2].any()
