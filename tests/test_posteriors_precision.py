"""The row operators where a loose tolerance would hide a mistake: low temperatures."""
import numpy as np
import pytest
import torch


U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from soft_clustering_em_b200 import build
    from soft_clustering_em_b200 import gmm

    build.build()
    gmm.load_library()
    return gmm


def _place(x, dtype, pad=0, shift=0):
    """x in rows of K + pad, `shift` entries into a buffer of NaN, and its values as float32."""
    N, K = x.shape
    t = DTYPES[dtype]
    buf = torch.full((N * (K + pad) + shift + 64,), float("nan"), dtype=t, device="cuda")
    Z = buf[shift:shift + N * (K + pad)].view(N, K + pad)[:, :K]
    Z.copy_(torch.from_numpy(x))
    return Z, Z.float().cpu().numpy()


# ------------------------------------------------------------------ low temperatures
# The exponent t of a class is at most 32 in size for the classes that count (a thread's reference
# is raised when its sum passes 2^20): 2^-20 for its rounding, as much for moving a sum to another
# reference and for the sum's logarithm, 2^-22 twice for the exponentials, (K / 256 + 64) u for the
# sum, all times log 2 or less.
def _lp_tol(K):
    return 4 * 2.0 ** -20 + (K / 256 + 64) * U


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, 1 / 0.07, 10.0, 100.0])
@pytest.mark.parametrize("K", [200, 1000, 1025, 5000, 70_001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_dominant_class_at_a_low_temperature(G, dtype, K, scale):
    """log p stays at or below 0 and a weight at or below 1, and both as near to them as they are."""
    rng = np.random.default_rng(K)
    x = rng.normal(size=(64, K)).astype(np.float32) * 2
    x[:, 17] = np.linspace(24, 60, 64)
    Z, v = _place(x, dtype)
    ids = torch.full((64,), 17, dtype=torch.int32, device="cuda")
    z = v.astype(np.float64) * np.float64(np.float32(scale))
    rest = np.delete(z, 17, 1) - z[:, 17:18]
    want = -np.log1p(np.exp(rest).sum(1))
    for m in (0, 2):
        r = G.gmm_logprobs(Z, ids, m=m, scale=scale)
        got = [r.logp] + ([r.top_logp[:, 0]] if m else [])
        for g in got:
            g = g.double().cpu().numpy()
            assert (g <= 0).all(), g.max()
            # (the rest's exponents are off by 2^-22 of their size, at most 104 where they count)
            tol = _lp_tol(K) + np.abs(want) * 104 * 2.0 ** -22
            assert (np.abs(g - want) <= tol).all(), np.abs(g - want).max()
    for renorm in (False, True):
        _, w = G.gmm_route(Z, 2, renorm=renorm, scale=scale)
        assert w.max().item() <= (1 + 8 * U if renorm else 1)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, 0.3, 1 / 0.07, 100.0])
@pytest.mark.parametrize("K", [40, 900, 1500, 33_000])
def test_probabilities_sum_to_one_at_a_low_temperature(G, K, scale):
    """Twenty classes side by side far from 0 and the others masked: their p's sum to 1."""
    rng = np.random.default_rng(K)
    N = 64
    x = np.full((N, K), -np.inf, np.float32)
    for n in range(N):
        x[n, rng.permutation(K)[:20]] = 50 + n / 8 + rng.random(20) * 3 / max(1.0, scale)
    Z, v = _place(x, "f32", 3)
    r = G.gmm_logprobs(Z, m=20, scale=scale)
    p = r.top_logp.double().exp().sum(1).cpu().numpy()
    assert (np.abs(p - 1) <= _lp_tol(K)).all(), np.abs(p - 1).max()
    if K <= 1000:
        for renorm in (False, True):
            idx, w = G.gmm_route(Z, 8, renorm=renorm, scale=scale)
            lp = r.top_logp[:, :8].double()
            want = (lp.softmax(1) if renorm else lp.exp()).cpu().numpy()
            assert (np.abs(w.double().cpu().numpy() - want) <= want * 2 * _lp_tol(K)).all()
