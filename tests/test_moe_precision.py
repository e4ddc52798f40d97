"""How exactly gmm_moe keeps the inner activations: small and large ones, both types, against the
2-norm limit of oracle/posteriors.py, and mistakes planted in a restatement on the CPU."""
import numpy as np
import pytest
import torch

from oracle import posteriors as P

TYPES = ("bf16", "f16")
# tokens' scale, W_down's gain
SCALES = [(1.0, 1.0), (8.0, 1.0), (0.1, 1.0), (0.01, 10.0), (0.003, 10.0), (0.001, 100.0)]
T, E, D, F, M = 24, 3, 64, 256, 2
CANCEL = [1.0, 2.0 ** -8, 2.0 ** -12]


def _case(dtype, size, gain):
    """Values of the type, as float64 (numpy), that a layer of this scale has."""
    rng = np.random.default_rng(int(size * 1000) + int(gain))
    X = P.to_type(rng.normal(size=(T, D)) * size, dtype)
    W_up = P.to_type(rng.normal(size=(E, 2 * F, D)) / np.sqrt(D), dtype)
    W_down = P.to_type(rng.normal(size=(E, D, F)) / np.sqrt(F) * gain, dtype)
    idx = np.stack([rng.permutation(E)[:M] for _ in range(T)]).astype(np.int32)
    resp = rng.random((T, M)).astype(np.float32)
    return X, idx, resp, W_up, W_down


def _halves(h, dtype, lo_scale):
    """h as the pair keeps it, with lo times lo_scale (0: no lo)."""
    hi = P.to_type(h, dtype)
    return hi + (P.to_type((h - hi) * lo_scale, dtype) / lo_scale if lo_scale else 0.0)


def _restated(X, idx, resp, W_up, W_down, dtype, lo_scale):
    F = W_down.shape[2]
    Y = np.zeros(X.shape)
    for t in range(len(X)):
        for e, w in zip(idx[t], resp[t].astype(np.float64)):
            up = W_up[e] @ X[t]
            Y[t] += w * (W_down[e] @ _halves(P.activation(up[:F], 0) * up[F:], dtype, lo_scale))
    return P.to_type(Y, dtype)


def _over(Y, want, limit):
    return np.linalg.norm(Y - want, axis=1) > limit


def _cancelling(dtype, size):
    """(case, y, tolerance): y = h_1 - h_0 of two activations that differ by less than the type
    resolves.  Both gates are 32, far enough out that silu(32) = 32 in float32, so y is what the lo
    halves keep: u / 4 of h for half a step u of the type."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    X = np.zeros((1, 8))
    X[0, :3] = 32.0, size, size * u
    W_up = np.zeros((1, 16, 8))
    W_up[0, :2, 0] = 1.0             # gates
    W_up[0, 8:10, 1] = 1.0 + 2 * u   # linear: size (1 + 2 u), the second size u / 4 more
    W_up[0, 9, 2] = 0.25
    W_down = np.zeros((1, 8, 8))
    W_down[0, :, 0], W_down[0, :, 1] = -1.0, 1.0
    want = 32 * size * u / 4
    tol = 2 * 32 * size * (1 + 3 * u) * (2.0 ** -17 if dtype == "bf16" else 2.0 ** -22) + want * u
    return (X, np.zeros((1, 1), np.int32), np.ones((1, 1), np.float32), W_up, W_down), want, tol


def _good(dtype):
    return 2.0 ** 11 if dtype == "f16" else 1.0


@pytest.mark.parametrize("size,gain", SCALES)
@pytest.mark.parametrize("dtype", TYPES)
def test_planted_mistakes_are_seen(dtype, size, gain):
    """A pair within its stated precision passes.  A bf16 one without its lo half does not (fp16:
    the next test), nor, where the activations are small, an fp16 lo half that underflows."""
    c = _case(dtype, size, gain)
    want, limit = P.moe_limit(*c, 0, dtype)
    assert not _over(_restated(*c, dtype, _good(dtype)), want, limit).any()
    if dtype == "bf16":
        assert _over(_restated(*c, dtype, 0.0), want, limit).any()
    elif size <= 0.003:
        assert _over(_restated(*c, dtype, 1.0), want, limit).any()


@pytest.mark.parametrize("size", CANCEL)
@pytest.mark.parametrize("dtype", TYPES)
def test_a_lost_low_half_is_seen(dtype, size):
    c, want, tol = _cancelling(dtype, size)
    assert np.abs(_restated(*c, dtype, _good(dtype)) - want).max() <= tol
    assert np.abs(_restated(*c, dtype, 0.0) - want).max() > tol


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from soft_clustering_em_b200 import build
    from soft_clustering_em_b200 import gmm

    build.build()
    gmm.load_library()
    return gmm


def _gpu(dtype, X, idx, resp, W_up, W_down):
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    X, W_up, W_down = (torch.from_numpy(v).cuda().to(t) for v in (X, W_up, W_down))
    return X, torch.from_numpy(idx).cuda(), torch.from_numpy(resp).cuda(), W_up, W_down


@pytest.mark.gpu
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("size,gain", SCALES)
@pytest.mark.parametrize("dtype", TYPES)
def test_activations_of_every_size(G, dtype, size, gain, act):
    c = _case(dtype, size, gain)
    want, limit = P.moe_limit(*c, act, dtype)
    Y = G.gmm_moe(*_gpu(dtype, *c), act=act).double().cpu().numpy()
    off = np.linalg.norm(Y - want, axis=1)
    assert (off <= limit).all(), float((off / limit).max())


@pytest.mark.gpu
@pytest.mark.parametrize("size", CANCEL)
@pytest.mark.parametrize("dtype", TYPES)
def test_what_is_left_where_the_high_halves_cancel(G, dtype, size):
    c, want, tol = _cancelling(dtype, size)
    Y = G.gmm_moe(*_gpu(dtype, *c)).double().cpu().numpy()
    assert (np.abs(Y - want) <= tol).all(), (Y, want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
def test_activations_far_below_zero(G, dtype, act):
    """An activation's own error, by itself: one gate value per expert, 2^10 beside and behind it.
    The exponent, at most 40, is off by 2^-21 in relation, so its power by 2^-15; h by 2^-17 or, in
    fp16 below 2^-14, by 2^-36."""
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    v = np.arange(-7.0, 7.25, 0.25)  # (each of the type)
    n = len(v)
    W_up = torch.zeros(n, 16, 8, dtype=t, device="cuda")
    W_up[:, :8, 0] = torch.from_numpy(v).to(t).cuda()[:, None]
    W_up[:, 8:, 0] = 1024.0
    W_down = torch.zeros(n, 8, 8, dtype=t, device="cuda")
    W_down[:, 0, 0] = 8.0
    X = torch.zeros(n, 8, dtype=t, device="cuda")
    X[:, 0] = 1.0
    idx = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    resp = torch.ones(n, 1, device="cuda")
    Y = G.gmm_moe(X, idx, resp, W_up, W_down, act=act)[:, 0].double().cpu().numpy()
    want = P.activation(v, act) * 8192
    f = torch.finfo(t)
    tol = np.abs(want) * (f.eps / 2 + 2.0 ** -15 + 2.0 ** -17) + 8 * 2.0 ** -36
    tol = tol + f.smallest_normal * f.eps / 2
    assert (np.abs(Y - want) <= tol).all(), (v[np.abs(Y - want) > tol], np.max(np.abs(Y - want) / tol))
