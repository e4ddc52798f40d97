"""Pins of oracle/posteriors.py (CPU): closed forms, differences, and an independent restatement."""
import numpy as np
import pytest

from oracle import posteriors as P


def test_two_classes_by_hand():
    # logits 0 and log 3: p = 1/4, 3/4
    x = np.array([[0.0, np.log(3.0)]], np.float32)
    logp, H, lse, idx, top = P.logprobs(x, np.array([0]), 2)
    assert logp[0] == pytest.approx(np.log(0.25), abs=1e-7)
    assert H[0] == pytest.approx(-(0.25 * np.log(0.25) + 0.75 * np.log(0.75)), abs=1e-7)
    assert lse[0] == pytest.approx(np.log(4.0), abs=1e-7)
    assert idx.tolist() == [[1, 0]]
    np.testing.assert_allclose(np.exp(top), [[0.75, 0.25]], atol=1e-7)


def test_rows_sum_to_one_and_uniform_entropy():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 17)).astype(np.float32) * 4
    _, _, _, _, top = P.logprobs(x, None, 17)
    np.testing.assert_allclose(np.exp(top).sum(1), 1.0, atol=1e-12)
    _, H, _, idx, _ = P.logprobs(np.full((1, 8), 3.0, np.float32), None, 4, scale=0.5)
    assert H[0] == pytest.approx(np.log(8.0)) and idx.tolist() == [[0, 1, 2, 3]]  # ties in order


def test_masked_empty_and_bad_rows():
    inf = np.inf
    x = np.array([[-inf, 1.0, -inf], [-inf] * 3, [0.0, np.nan, 1.0], [0.0, inf, 1.0]], np.float32)
    logp, H, lse, idx, top = P.logprobs(x, np.array([1, 0, 0, -1]), 2)
    assert logp[0] == 0.0 and H[0] == 0.0 and lse[0] == 1.0
    assert idx.tolist() == [[1, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert logp[1] == -inf and H[1] == 0.0 and lse[1] == -inf and (top[1] == -inf).all()
    assert np.isnan(logp[2]) and np.isnan(H[2]) and np.isnan(lse[3]) and logp[3] == 0.0
    gi, gr = P.route(x, 2, True)
    assert gr[0].tolist() == [1.0, 0.0] and gr[1].tolist() == [0.0, 0.0]


@pytest.mark.parametrize("scale", [1.0, 0.75])
def test_gradient_against_differences(scale):
    rng = np.random.default_rng(1)
    N, K, m = 3, 9, 3
    # float32 values on a grid of 1/64, so that steps of 1/64 stay exact in float32
    x = (np.round(rng.normal(size=(N, K)) * 64) / 64).astype(np.float32)
    x[1, 4] = -np.inf
    ids = np.array([2, 0, -1])
    top_idx = P.logprobs(x, ids, m, scale)[3]
    w = [rng.normal(size=s) for s in ((N,), (N,), (N,), (N, m))]

    def value(x):
        z = x.astype(np.float64) * np.float64(np.float32(scale))
        lse = np.log(np.exp(z).sum(1))
        lp = z - lse[:, None]
        p = np.exp(lp)
        H = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(1)
        use = ids >= 0
        out = (w[0] * np.where(use, lp[np.arange(N), np.maximum(ids, 0)], 0)).sum()
        out += (w[1] * H).sum() + (w[2] * lse).sum()
        return out + (w[3] * np.take_along_axis(lp, top_idx, 1)).sum()

    z = P.logits(x, scale)
    _, _, lse = P._rowwise(z)
    H = P.logprobs(x, None, 0, scale)[1]
    g = P.gradient(x, ids, lse, H, w[0], w[1], w[2], top_idx, w[3], scale)
    assert g[1, 4] == 0.0
    step = 1.0 / 1024
    for n in range(N):
        for k in range(K):
            if not np.isfinite(x[n, k]):
                continue
            hi, lo = x.copy(), x.copy()
            hi[n, k] += step
            lo[n, k] -= step
            # third derivatives of these sums are below 40: step^2 / 6 of that is 7e-6
            assert (value(hi) - value(lo)) / (2 * step) == pytest.approx(g[n, k], abs=1e-5)


def test_gradient_of_an_empty_row_is_zero_and_named_twice_adds():
    x = np.full((1, 4), -np.inf, np.float32)
    g = P.gradient(x, np.array([1]), np.array([-np.inf]), np.zeros(1), np.ones(1), np.ones(1),
                   np.ones(1), None, None)
    assert (g == 0).all()
    x = np.zeros((1, 2), np.float32)
    lse = np.array([np.log(2.0)])
    g = P.gradient(x, np.array([0]), lse, None, np.ones(1), None, None, np.array([[0, 0]]),
                   np.array([[1.0, 1.0]]))
    np.testing.assert_allclose(g, [[1.5, -1.5]])


@pytest.mark.parametrize("act", [0, 1])
def test_moe_against_a_dense_restatement(act):
    import torch

    rng = np.random.default_rng(2)
    T, D, F, E, m = 5, 8, 16, 4, 3
    X, U, W = rng.normal(size=(T, D)), rng.normal(size=(E, 2 * F, D)), rng.normal(size=(E, D, F))
    idx = rng.integers(-1, E, size=(T, m)).astype(np.int32)
    resp = rng.random((T, m))
    Y, bound = P.moe(X, idx, resp, U, W, act)
    G = np.zeros((T, E))
    for t in range(T):
        for j in range(m):
            if idx[t, j] >= 0:
                G[t, idx[t, j]] += resp[t, j]
    x, u, w = (torch.from_numpy(a) for a in (X, U, W))
    up = torch.einsum("td,efd->tef", x, u)
    fn = torch.nn.functional.silu if act == 0 else (
        lambda v: torch.nn.functional.gelu(v, approximate="tanh"))
    ref = torch.einsum("te,tef,edf->td", torch.from_numpy(G), fn(up[..., :F]) * up[..., F:], w)
    np.testing.assert_allclose(Y, ref.numpy(), rtol=1e-12, atol=1e-12)
    assert (bound >= np.abs(Y) - 1e-12).all()


def test_planted_mistakes_in_the_order_are_caught():
    z = np.array([[1.0, 2.0, 2.0, -np.inf]])
    assert P.order(z, 4).tolist() == [[1, 2, 0, -1]]
    higher_first = np.argsort(-z[0][::-1], kind="stable")  # ties to the higher index
    assert (3 - higher_first)[:2].tolist() != P.order(z, 4)[0, :2].tolist()
