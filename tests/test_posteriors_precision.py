"""The row operators where a loose tolerance would hide a mistake: low temperatures, rows far from
0, and every entry of the gradient by itself.  Against oracle/posteriors.py, which also says how
the limits come about."""
import numpy as np
import pytest
import torch

from oracle import posteriors as P

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


# ------------------------------------------------------------------ the gradient
def _upstream(rng, N, m):
    up = {k: rng.normal(size=N).astype(np.float32) for k in ("dlogp", "dentropy", "dlse")}
    up["dtop"] = rng.normal(size=(N, m)).astype(np.float32) if m else None
    return up


def _limit(x, ids, lse, H, up, idx, scale, dtype):
    f = torch.finfo(DTYPES[dtype])
    return P.gradient_limit(x, ids, lse, H, up["dlogp"], up["dentropy"], up["dlse"], idx,
                            up["dtop"], scale, f.eps, f.smallest_normal)


def _check(G, Z, x, ids, m, scale, dtype, out=None, seed=0):
    up = _upstream(np.random.default_rng(seed), len(x), m)
    ids_d = torch.from_numpy(ids).cuda()
    r = G.gmm_logprobs(Z, ids_d, m=m, scale=scale)
    idx = r.top_idx.cpu().numpy() if m else None
    want, tol = _limit(x, ids, r.lse.cpu().numpy(), r.entropy.cpu().numpy(), up, idx, scale, dtype)
    d = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in up.items()}
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = G.gmm_logprobs_backward(Z, ids_d, r.lse, entropy=r.entropy, top_idx=r.top_idx,
                                  scale=scale, out=out, dev_flags=flags, **d)
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4],
                           tol[bad][:4])
    assert flags.item() == 0
    return got


def _logits(rng, N, K):
    x = rng.normal(size=(N, K)).astype(np.float32) * 3
    x[np.arange(N), rng.integers(0, K, N)] += 8
    return x


@pytest.mark.parametrize("m", [0, 5, 32])
@pytest.mark.parametrize("K", [40, 1001, 2049, 8192, 33_000, 131_072])
def test_lost_and_turned_entries_of_the_gradient_are_seen(K, m):
    """Of the entries that no label and no alternative names, a limit lets hardly one pass as 0 or
    with its sign turned (those whose terms happen to cancel)."""
    rng = np.random.default_rng(K)
    x = _logits(rng, 3, K)
    ids = rng.integers(0, K, 3).astype(np.int32)
    _, H, lse, idx, _ = P.logprobs(x, ids, m)
    up = _upstream(rng, 3, m)
    for dtype in DTYPES:
        want, tol = _limit(x, ids, lse, H, up, idx if m else None, 1.0, dtype)
        free = np.ones(x.shape, bool)
        free[np.arange(3), ids] = False
        if m:
            np.put_along_axis(free, idx.astype(np.int64), False, 1)
        # (fp16: what is below its smallest numbers is 0)
        free &= np.abs(want) > 2 * torch.finfo(DTYPES[dtype]).smallest_normal
        assert free.sum() > 0
        for wrong in (np.zeros_like(want), -want):
            assert (np.abs(wrong - want) > tol)[free].mean() > 0.99


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("K", [1, 3, 8, 33, 256, 1001, 2048, 2049, 8192, 33_000, 131_072])
def test_every_entry_of_the_gradient(G, K, dtype):
    rng = np.random.default_rng(K)
    N = 23 if K < 20_000 else 3
    for pad, shift, m, scale, masked in ((0, 0, 0, 1.0, False), (3, 1, 5, 0.75, True),
                                         (8, 0, 32, 1.25, False)):
        x = _logits(rng, N, K)
        if masked:
            x[rng.random((N, K)) < 0.4] = -np.inf
            x[2] = -np.inf
        Z, v = _place(x, dtype, pad, shift)
        ids = rng.integers(0, K, N).astype(np.int32)
        ids[1::4] = -1
        _check(G, Z, v, ids, m, scale, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("K", [1, 7, 300, 2048, 2049, 9000, 40_003])
def test_gradient_of_rows_far_from_zero(G, K, dtype):
    """Rows whose log-sum-exp rounds away what p needs: the type's lowest value as a mask that
    leaves nothing else, log-joints in the thousands, and rows of ordinary size among them."""
    t = DTYPES[dtype]
    rng = np.random.default_rng(K)
    low = float(torch.finfo(t).min)
    bases = [low, -60_000.0, 30_000.0, -1500.0, 1100.0, 0.0, -5.0, low, -2000.0]
    if dtype != "f16":
        bases += [-1e30, 1e30, 3e38, -1e20]
    x = np.array(bases, np.float32)[:, None] + _logits(rng, len(bases), K)
    x[0] = low
    x[4, rng.random(K) < 0.5] = -np.inf
    x[7, rng.random(K) < 0.5] = -np.inf  # some masked either way
    x[8, K // 2:] = low
    x[4, K // 2] = 1100.0
    x[7, K // 2] = low
    Z, v = _place(np.maximum(x, low, where=x > -np.inf, out=x), dtype, 3, 1)
    ids = rng.integers(0, K, len(bases)).astype(np.int32)
    ids[3] = -1
    for m, scale in ((0, 1.0), (min(5, K), 0.5), (3, 2.0 if dtype == "f16" else 1.0)):
        got = _check(G, Z, v, ids, m, scale, dtype, seed=m).clone()
        W, w = _place(v, dtype, 3, 1)
        same = _check(G, W, w, ids, m, scale, dtype, out=W, seed=m)  # in place
        assert torch.equal(got, same)
