"""oracle/assignments.py against differences and against itself in other words (no GPU)."""
import numpy as np
import pytest

from oracle import assignments as A
from oracle import posteriors as P


def _difference(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("m,weights", [(1, False), (3, True)])
def test_embed_gradients_are_differences(m, weights):
    rng = np.random.default_rng(1)
    K, D, N = 5, 3, 7
    W, dY = rng.normal(size=(K, D)), rng.normal(size=(N, D))
    idx = rng.integers(-1, K, (N, m))
    idx[0, 0] = K  # left out
    r = rng.normal(size=(N, m)) if weights else None

    def value(W, r):
        return (A.embed(W, idx, r, 1.5)[0] * dY).sum()

    dW, size, named = A.embed_backward(dY, idx, K, r, 1.5)
    np.testing.assert_allclose(dW, _difference(lambda w: value(w, r), W), atol=1e-8)
    assert named.sum() == ((idx >= 0) & (idx < K)).sum() and (size >= np.abs(dW) - 1e-12).all()
    if weights:
        d, _ = A.embed_dresp(dY, W, idx, 1.5)
        np.testing.assert_allclose(d, _difference(lambda q: value(W, q), r), atol=1e-8)


def _route_value(x, idx, renorm, dresp, db, dz, counts, rows, offsets, mask, scale):
    """The function whose gradient route_backward is, with the counts held fixed, from softmax."""
    z = x * np.float64(np.float32(scale))
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    total = 0.0
    for n in range(len(x)):
        ks = [(j, k) for j, k in enumerate(idx[n]) if k >= 0]
        denominator = sum(p[n, k] for _, k in ks) if renorm else 1.0
        total += sum(dresp[n, j] * p[n, k] / denominator for j, k in ks)
    o = [0, len(x)] if offsets is None else offsets
    K, m = x.shape[1], idx.shape[1]
    for s in range(len(o) - 1):
        n = [i for i in range(o[s], o[s + 1]) if mask is None or mask[i]]
        if n:
            f = counts[s] / (m * len(n))
            total += db[s] * K * (f * p[n].mean(0)).sum() + dz[s] * (lse[n] ** 2).mean()
    return total


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_route_gradient_is_a_difference(renorm, packed):
    rng = np.random.default_rng(2)
    N, K, m = 9, 5, 2
    x = rng.normal(size=(N, K))
    idx = P.order(x, m)
    idx[2, 1] = -1
    offsets = [0, 3, 3, 7] if packed else None
    mask = rng.random(N) < 0.7 if packed else None
    S = 3 if packed else 1
    _, _, load, counts, rows = A.route_loss(x, idx, offsets, mask, 0.75)
    dresp, db, dz = rng.normal(size=(N, m)), rng.normal(size=S), rng.normal(size=S)
    got, size = A.route_backward(x, idx, dresp, renorm, counts, rows, db, dz, offsets, mask, 0.75)
    want = _difference(lambda y: _route_value(y, idx, renorm, dresp, db, dz, counts, rows, offsets,
                                              mask, 0.75), x)
    np.testing.assert_allclose(got, want, atol=1e-8)
    assert (size >= np.abs(got) - 1e-12).all()
    if not packed:
        assert abs(load.sum() - 1) < 1e-12 and counts.sum() == (idx >= 0).sum()


def test_an_even_load_has_a_balance_of_one():
    x = np.zeros((8, 4))
    idx = np.array([[i % 4, (i + 1) % 4] for i in range(8)])
    balance, z, load, counts, rows = A.route_loss(x, idx)
    assert abs(balance[0] - 1) < 1e-12 and (counts == 4).all() and rows[0] == 8
    assert abs(z[0] - np.log(4) ** 2) < 1e-12


def test_beams_are_searched_in_order():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]))
    s, p, t = A.beam_select(x, [[0.0, -0.1]], 4)
    assert p.tolist() == [[1, 0, 0, 0]] and t.tolist() == [[1, 0, 1, 2]]
    s, p, t = A.beam_select(x, [[0.0, -np.inf]], 4)
    assert p.tolist() == [[0, 0, 0, -1]] and s[0, 3] == -np.inf
    s, p, t = A.beam_select(x, [[-1.0, -0.1]], 3, ended=[[0, 1]], end_id=2)
    assert p.tolist() == [[1, 0, 0]] and t.tolist() == [[2, 0, 1]] and s[0, 0] == -0.1


def test_states_follow_their_parents():
    state = np.arange(4 * 3 * 2).reshape(4, 3, 2)
    got = A.beam_reorder(state, np.array([[1, 0], [1, -1]]), np.array([2, 3]), 1)
    assert (got[0, :2] == state[1, :2]).all() and (got[0, 2] == state[0, 2]).all()
    assert (got[1, :2] == state[0, :2]).all()
    assert (got[2] == state[3]).all() and (got[3] == state[3]).all()
