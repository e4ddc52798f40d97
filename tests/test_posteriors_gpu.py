"""gmm_logprobs, its gradient and gmm_route on the GPU against oracle/posteriors.py.

Tolerances, for u = 2^-24 (half a step of float32):
  z is exact (the oracle rounds it too); d = z - M is off by at most u (|z| + |M| + |d|)
  (the product is rounded in the maximum and not in the difference), e^d in relation by that,
  by 2 u |d| (the product with log2 e and that constant) and by 2^-22 (the hardware exponential);
  a sum of c terms one after another and ten levels of merging adds (c + 30) u.  A row's weight
  is in its largest terms: |d| <= 104 wherever e^d is not 0, so
     rel(S) <= u (2 max|z| + 3 * 104 + c + 34) =: s
  and log p, lse and H = log S - U / S are off by at most that much plus their own roundings:
     |lse|, |log p|: s + 4 u (|z| + |M| + |log p|);   H: s (2 + H) + 8 u (1 + H).
  c is at most the classes a thread adds up: K / 256 rounded up, plus 40.
Gradient: lse is given, log p off by u (|z| + |lse| + |log p|), p in relation by that plus
3 u |log p| + 2^-22, the sum in brackets by 4 u times its terms' magnitudes; then half a step of
the type on the whole.
"""
import numpy as np
import pytest

from oracle import posteriors as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ("f32", "bf16", "f16")


@pytest.fixture(scope="module")
def G():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from soft_clustering_em_b200 import build
    from soft_clustering_em_b200 import gmm

    build.build()
    gmm.load_library()
    return gmm


def _t(dtype):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def _place(x, dtype, pad=0, shift=0):
    """x (float32 array) on the GPU in rows of K + pad, starting `shift` entries into a buffer
    whose other entries are NaN; returns the view and its values as float32."""
    import torch

    N, K = x.shape
    buf = torch.full((N * (K + pad) + shift + 64,), float("nan"), dtype=_t(dtype), device="cuda")
    Z = buf[shift:shift + N * (K + pad)].view(N, K + pad)[:, :K]
    Z.copy_(torch.from_numpy(x))
    return Z, Z.float().cpu().numpy()


def _tols(x, lse, lp, H, scale):
    z = P.logits(x, scale)
    size = np.where(np.isfinite(z), np.abs(z), 0.0).max(1)
    size = np.minimum(size, 1e30)
    s = U * (2 * size + 3 * 104 + x.shape[1] / 256 + 41 + 34)
    own = 4 * U * (2 * size[:, None] + np.where(np.isfinite(lp), np.abs(lp), 0.0))
    return s, s[:, None] + own, s * (2 + H) + 8 * U * (1 + H)


def _near(got, want, tol, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = np.broadcast_to(tol, want.shape)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine], err_msg=what)  # nan equals nan here
    bad = np.abs(got[fine] - want[fine]) > tol[fine]
    assert not bad.any(), (what, got[fine][bad][:4], want[fine][bad][:4], tol[fine][bad][:4])


def _check(G, Z, x, ids, m, scale):
    import torch

    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids_d = None if ids is None else torch.from_numpy(ids).cuda()
    r = G.gmm_logprobs(Z, ids_d, m=m, scale=scale, dev_flags=flags)
    logp, H, lse, idx, top = P.logprobs(x, ids, m, scale)
    with np.errstate(invalid="ignore"):
        s, lp_tol, H_tol = _tols(x, lse, np.concatenate([logp[:, None], top], 1), H, scale)
    _near(r.lse.cpu(), lse, lp_tol[:, 0], "lse")
    _near(r.entropy.cpu(), H, H_tol, "entropy")
    if ids is not None:
        _near(r.logp.cpu(), logp, lp_tol[:, 0], "logp")
    if m:
        np.testing.assert_array_equal(r.top_idx.cpu().numpy(), idx)
        _near(r.top_logp.cpu(), top, lp_tol[:, 1:], "top_logp")
    else:
        assert r.top_idx is None and r.top_logp is None
    return r, int(flags.item())


def _logits(rng, N, K, spread=3.0):
    x = rng.normal(size=(N, K)).astype(np.float32) * spread
    x[np.arange(N), rng.integers(0, K, N)] += 8
    return x


CLASSES = (1, 2, 5, 8, 31, 32, 33, 64, 100, 129, 255, 256, 257, 512, 513, 1000, 1023, 1024, 1025,
           1031, 2048, 2051, 8191, 40_009, 131_072)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", CLASSES)
def test_logprobs_sizes(G, K, dtype):
    rng = np.random.default_rng(K)
    N = 41 if K < 20_000 else 3
    for pad, shift, m, scale in ((0, 0, 5, 1.0), (3, 1, 20, 0.75), (8, 0, 0, 1.25)):
        Z, x = _place(_logits(rng, N, K), dtype, pad, shift)
        ids = rng.integers(0, K, N).astype(np.int32)
        ids[::5] = -1
        _, flags = _check(G, Z, x, ids, m, scale)
        assert flags == 0


@pytest.mark.parametrize("K", [7, 128, 200, 1000, 1500, 30_011])
@pytest.mark.parametrize("N", [1, 2, 37, 700, 5003])
def test_logprobs_row_counts(G, N, K):
    if N * K > 6_000_000:
        N = 6_000_000 // K
    rng = np.random.default_rng(N + K)
    Z, x = _place(_logits(rng, N, K), "bf16", 1)
    _check(G, Z, x, rng.integers(0, K, N).astype(np.int32), 3, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [9, 300, 1024, 5000, 70_001])
def test_masks_ties_and_orders(G, K, dtype):
    import torch

    rng = np.random.default_rng(K + 1)
    low = float(torch.finfo(_t(dtype)).min)
    inf = np.inf
    x = np.round(_logits(rng, 20, K))  # whole numbers: many ties
    x[1] = 1.0                          # all equal
    x[2] = -inf
    x[3] = low                          # a mask by the type's lowest value leaves nothing else
    x[4, rng.random(K) < 0.7] = -inf
    x[5, rng.random(K) < 0.7] = low
    x[6] = -inf
    x[6, K - 1] = -2.0                  # one class left, the last
    x[7] = -inf
    x[7, 0] = low                       # one class left, at the lowest value
    x[8] = np.linspace(-30, 30, K)      # ascending
    x[9] = np.linspace(30, -30, K)      # descending
    x[10] = np.where(np.arange(K) % 2, 0.0, -0.0)  # both zeros are equal
    x[11, 3] = np.nan
    x[12, K // 2] = inf
    x[13] = low
    x[13, K // 3] = -5.0
    x[14] = -inf
    x[14, ::max(1, K // 3)] = 4.0       # a few tied classes, the rest masked
    x[15, :] = 200.0                    # large, equal
    x[15, 0] = 60.0
    ids = rng.integers(0, K, 20).astype(np.int32)
    ids[13], ids[6], ids[7], ids[16], ids[17] = K // 3, K - 1, 0, -1, K
    ids[18] = -7
    for pad, m, scale in ((0, 8, 1.0), (5, 32, 0.5), (2, 1, 1.0)):
        Z, v = _place(x, dtype, pad)
        _, flags = _check(G, Z, v, ids, m, scale)
        assert flags == G.GMM_DEVFLAG_NONFINITE_X | G.GMM_DEVFLAG_BAD_INDEX


def test_a_scaled_logit_that_overflows_is_masked_or_infinite(G):
    x = np.zeros((2, 2000), np.float32)
    x[0, 7] = np.finfo(np.float32).min
    x[1, 7] = np.finfo(np.float32).max
    Z, v = _place(x, "f32")
    r, flags = _check(G, Z, v, np.array([7, 7], np.int32), 2, 2.0)
    assert r.logp[0].item() == -np.inf and np.isnan(r.logp[1].item())
    assert flags == G.GMM_DEVFLAG_NONFINITE_X


@pytest.mark.parametrize("m", [1, 2, 7, 31, 32])
@pytest.mark.parametrize("K", [33, 1200, 9001])
def test_alternatives_where_one_thread_holds_them_all(G, K, m):
    """The best classes side by side, a vector apart and a whole batch of threads apart."""
    for step in (1, 4, 8, 256, 1024, 2048):
        x = np.random.default_rng(m).normal(size=(4, K)).astype(np.float32)
        x[0, ::step][:40] += 50
        x[1, ::-step][:40] += 50
        x[2, ::step][:40] = 60
        Z, v = _place(x, "bf16")
        _check(G, Z, v, None, m, 1.0)


def test_the_most_classes(G):
    """2^24 classes, with ties at the top and masked stretches."""
    K = 1 << 24
    rng = np.random.default_rng(8)
    x = rng.integers(-40, 9, size=(2, K)).astype(np.float32)
    x[0, 1000:9000] = -np.inf
    x[1, K - 3], x[1, 77] = 12.0, 12.0
    Z, v = _place(x, "bf16", 3, 1)
    _check(G, Z, v, np.array([5, K - 1], np.int32), 7, 1.0)
    Zg = Z[:, :1 << 20]
    _grad_check(G, Zg, v[:, :1 << 20], np.array([5, 77], np.int32), 3, 1.0)


def test_rows_that_only_a_stretch_is_left_of(G):
    """A mask that leaves one stretch of classes: whole warps and CTAs see nothing."""
    K = 50_000
    for lo, hi in ((0, 40), (25_000, 25_300), (K - 9, K), (49_000, 49_001)):
        x = np.full((3, K), -np.inf, np.float32)
        x[:, lo:hi] = np.random.default_rng(lo).normal(size=(3, hi - lo)) * 30 - 500
        for dtype in ("f32", "bf16"):
            Z, v = _place(x, dtype, 1)
            _check(G, Z, v, np.array([lo, hi - 1, 0], np.int32), 32, 1.0)


def test_rising_and_falling_logits(G):
    """The reference has to follow: rows that rise by hundreds of powers of two, and fall."""
    K = 40_000
    ramp = np.linspace(-30_000, 30_000, K).astype(np.float32)
    x = np.stack([ramp, -ramp, np.abs(ramp), -np.abs(ramp), np.roll(ramp, K // 3)])
    for dtype in TYPES:
        Z, v = _place(x, dtype)
        _check(G, Z, v, np.array([K - 1, 0, 3, K // 2, 9], np.int32), 6, 1.0)
        _check(G, Z, v, np.array([K - 1, 0, 3, K // 2, 9], np.int32), 0, 0.5)


def _grad_case(rng, K, N, m, dtype, pad, shift, masked):
    x = _logits(rng, N, K)
    if masked:
        x[rng.random((N, K)) < 0.4] = -np.inf
        x[2] = -np.inf
    Z, v = _place(x, dtype, pad, shift)
    ids = rng.integers(0, K, N).astype(np.int32)
    ids[1::4] = -1
    return Z, v, ids


def _grad_check(G, Z, x, ids, m, scale, use=("dlogp", "dentropy", "dlse", "dtop"), out=None,
                top_idx=None, rng=None):
    import torch

    N, K = x.shape
    rng = rng or np.random.default_rng(5)
    r = G.gmm_logprobs(Z, None if ids is None else torch.from_numpy(ids).cuda(), m=m, scale=scale)
    lse, H = r.lse.cpu().numpy(), r.entropy.cpu().numpy()
    up = {k: rng.normal(size=N).astype(np.float32) if k in use else None
          for k in ("dlogp", "dentropy", "dlse")}
    up["dtop"] = rng.normal(size=(N, m)).astype(np.float32) if m and "dtop" in use else None
    idx = None
    if up["dtop"] is not None:
        idx = r.top_idx if top_idx is None else torch.from_numpy(top_idx).cuda()
    d = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in up.items()}
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = G.gmm_logprobs_backward(Z, None if ids is None else torch.from_numpy(ids).cuda(), r.lse,
                                  entropy=r.entropy, top_idx=idx, scale=scale, out=out,
                                  dev_flags=flags, **d)
    want = P.gradient(x, ids, lse, H, up["dlogp"], up["dentropy"], up["dlse"],
                      None if idx is None else idx.cpu().numpy(), up["dtop"], scale)
    z = P.logits(x, scale)
    ok = np.isfinite(z) & np.isfinite(lse)[:, None]
    zz, ll = np.where(ok, z, 0.0), np.where(np.isfinite(lse), lse, 0.0)[:, None]
    lp = np.where(ok, zz - ll, -200.0)
    p = np.exp(np.minimum(lp, 0.1))
    mag = sum(np.abs(up[k]) for k in ("dlogp", "dlse") if up[k] is not None)
    mag = mag + np.zeros(N)
    if up["dtop"] is not None:
        mag = mag + np.abs(up["dtop"]).sum(1)
    h = np.zeros(N) if up["dentropy"] is None else np.abs(up["dentropy"])
    terms = mag[:, None] + h[:, None] * (np.abs(lp) + np.abs(H)[:, None])
    off_lp = U * (np.abs(zz) + np.abs(ll) + np.abs(lp))
    rel_p = off_lp + 3 * U * np.abs(lp) + 2.0 ** -22
    tol = scale * p * (terms * (rel_p + (8 + m) * U) + h[:, None] * off_lp)
    named = np.abs(want) * 4 * U + scale * mag[:, None] * (4 + m) * U * (np.abs(want) > 0)
    half = torch.finfo(Z.dtype).eps / 2
    least = torch.finfo(Z.dtype).smallest_normal * torch.finfo(Z.dtype).eps
    tol = (tol + named) * 1.01 + np.abs(want) * half + least
    _near(got.float().cpu().numpy(), want, tol, "gradient")
    return got, int(flags.item())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 3, 8, 33, 256, 1001, 2048, 2049, 8192, 33_000, 131_072])
def test_gradient_sizes(G, K, dtype):
    rng = np.random.default_rng(K)
    N = 23 if K < 20_000 else 3
    for pad, shift, m, scale, masked in ((0, 0, 0, 1.0, False), (3, 1, 5, 0.75, True),
                                         (8, 0, 32, 1.25, False)):
        m = min(m, 32)
        Z, x, ids = _grad_case(rng, K, N, m, dtype, pad, shift, masked)
        _, flags = _grad_check(G, Z, x, ids, m, scale, rng=rng)
        assert flags == 0


@pytest.mark.parametrize("use", [("dlogp",), ("dentropy",), ("dlse",), ("dtop",),
                                 ("dlogp", "dentropy")])
@pytest.mark.parametrize("K", [77, 4100])
def test_gradient_of_each_output_alone(G, K, use):
    rng = np.random.default_rng(3)
    Z, x, ids = _grad_case(rng, K, 9, 4, "f32", 0, 0, True)
    _grad_check(G, Z, x, ids, 4, 1.0, use=use)


@pytest.mark.parametrize("K", [50, 1500, 9000])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_in_place_and_between_strided_rows(G, K, dtype):
    import torch

    rng = np.random.default_rng(7)
    N, m = 12, 6
    for shift_out, pad_out in ((0, 0), (1, 3), (4, 8)):
        Z, x, ids = _grad_case(rng, K, N, m, dtype, 5, 1, True)
        buf = torch.full((N * (K + pad_out) + shift_out + 16,), 7.0, dtype=_t(dtype),
                         device="cuda")
        view = buf[shift_out:shift_out + N * (K + pad_out)].view(N, K + pad_out)
        got, _ = _grad_check(G, Z, x, ids, m, 0.75, out=view[:, :K],
                             rng=np.random.default_rng(1))
        assert (view[:, K:] == 7.0).all() and (buf[:shift_out] == 7.0).all()
        assert (buf[shift_out + N * (K + pad_out):] == 7.0).all()
        again = got.clone()
        inplace, _ = _grad_check(G, Z, x, ids, m, 0.75, out=Z, rng=np.random.default_rng(1))
        assert inplace.data_ptr() == Z.data_ptr()
        assert torch.equal(inplace, again)  # bit for bit what the separate output got


def test_gradient_of_named_twice_bad_and_invalid(G):
    rng = np.random.default_rng(9)
    for K in (40, 3001):
        Z, x, ids = _grad_case(rng, K, 8, 4, "f32", 0, 0, False)
        idx = rng.integers(0, K, (8, 4)).astype(np.int32)
        idx[0, :] = ids[0] = 5      # label and all alternatives the same class
        idx[1, 1] = -1
        _, flags = _grad_check(G, Z, x, ids, 4, 1.0, top_idx=idx)
        assert flags == 0
        idx[2, 2], idx[3, 0], ids[4] = K, -3, K + 5
        _, flags = _grad_check(G, Z, x, ids, 4, 1.0, top_idx=idx)
        assert flags == G.GMM_DEVFLAG_BAD_INDEX
        x[5, 0] = np.nan
        Z, x = _place(x, "f32")
        ids[4] = 0
        _grad_check(G, Z, x, ids, 4, 1.0, top_idx=np.maximum(np.minimum(idx, K - 1), 0))


def test_gradient_against_differences(G):
    """The gradient against central differences of the forward call itself."""
    import torch

    rng = np.random.default_rng(11)
    N, K, m, scale, step = 4, 1100, 3, 0.75, 2.0 ** -4
    x = (np.round(rng.normal(size=(N, K)) * 2 * 64) / 64).astype(np.float32)
    ids = rng.integers(0, K, N).astype(np.int32)
    ids_d = torch.from_numpy(ids).cuda()
    w = [torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda() for s in
         ((N,), (N,), (N,), (N, m))]
    Z, _ = _place(x, "f32")
    r = G.gmm_logprobs(Z, ids_d, m=m, scale=scale)
    g = G.gmm_logprobs_backward(Z, ids_d, r.lse, w[0], r.entropy, w[1], w[2], r.top_idx, w[3],
                                scale=scale).double()

    def value(Zs):
        q = G.gmm_logprobs(Zs, ids_d, scale=scale)
        lp = (Zs.gather(1, r.top_idx.long()) * scale).double() - q.lse.double()[:, None]
        return ((w[0] * q.logp + w[1] * q.entropy + w[2] * q.lse).double()
                + (w[3].double() * lp).sum(1))

    for k in [0, 5, 255, 256, K - 1] + [int(i) for i in ids]:
        hi, lo = Z.clone(), Z.clone()
        hi[:, k] += step
        lo[:, k] -= step
        diff = (value(hi) - value(lo)) / (2 * step)
        # each value is off by s = u (2 max|z| + 3 * 104 + K / 256 + 75) times its weight (H's
        # by 2 + H of that); the third derivative of these sums is below 10
        s = U * (2 * 12 + 3 * 104 + K / 256 + 75)
        weight = (w[0].abs() + w[1].abs() * (2 + r.entropy) + w[2].abs() + w[3].abs().sum(1))
        tol = weight.double() * s / step + 10 * step ** 2 / 6
        assert ((diff - g[:, k]).abs() <= tol).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [1, 2, 8, 33, 64, 128, 200, 256, 512, 1000, 1025, 6000])
def test_route(G, E, dtype, renorm):
    rng = np.random.default_rng(E)
    for N, pad in ((1, 0), (130, 3), (3000, 0)):
        m = int(min(E, rng.integers(1, 9)))
        x = np.round(_logits(rng, N, E, 1.5) * 4) / 4  # ties
        if N > 3:
            x[1] = -np.inf
            x[2, 1:] = -np.inf
            x[3, 0] = np.nan
        Z, v = _place(x, dtype, pad)
        idx, resp = G.gmm_route(Z, m, renorm=renorm)
        ridx, rresp = P.route(v, m, renorm)
        np.testing.assert_array_equal(idx.cpu().numpy(), ridx)
        # p in relation by the error of its log (see above), |z| below 32, and expf's 2 u
        tol = np.abs(rresp) * (U * (2 * 32 + 3 * 104 + E / 256 + 80 + 4 * 96))
        _near(resp.cpu(), rresp, tol + 1e-37, "resp")


def test_route_feeds_the_lists(G):
    import torch

    from oracle import ivf

    Z = torch.randn(5000, 96, device="cuda")
    idx, resp = G.gmm_route(Z, 3)
    off, ids = G.gmm_ivf_build(idx, resp, 96, 0.05)
    ref_off, ref_ids = ivf.ivf_lists(idx.cpu().numpy(), resp.cpu().numpy(), 96, 0.05)
    np.testing.assert_array_equal(off.cpu().numpy(), ref_off)
    np.testing.assert_array_equal(ids[:ref_off[-1]].cpu().numpy(), ref_ids)


def test_rows_more_than_32_bits_apart(G):
    """Rows whose last starts over 2^31 entries (and 2^32 bytes) behind the first."""
    import torch

    N, K, ld = 9, 1500, 1 << 28
    buf = torch.empty((N - 1) * ld + K, dtype=torch.bfloat16, device="cuda")
    Z = buf.as_strided((N, K), (ld, 1))
    rng = np.random.default_rng(2)
    Z.copy_(torch.from_numpy(_logits(rng, N, K)))
    x = Z.float().cpu().numpy()
    ids = rng.integers(0, K, N).astype(np.int32)
    _check(G, Z, x, ids, 4, 1.0)
    _grad_check(G, Z, x, ids, 4, 1.0, out=Z)


def test_results_repeat_bit_for_bit(G):
    import torch

    for N, K in ((3, 131_072), (300, 5000), (4000, 256)):
        Z = torch.randn(N, K, device="cuda").bfloat16()
        a, b = G.gmm_logprobs(Z, m=8), G.gmm_logprobs(Z, m=8)
        for u, v in zip(a[1:], b[1:]):
            assert torch.equal(u, v)


def test_side_stream_and_captured_graph(G):
    import torch

    K, N = 5003, 64
    Z = torch.randn(N, K, device="cuda")
    ids = torch.randint(K, (N,), device="cuda", dtype=torch.int32)
    w = torch.randn(N, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = G.gmm_logprobs(Z, ids, m=4)
        g = G.gmm_logprobs_backward(Z, ids, r.lse, dlogp=w)
    side.synchronize()
    assert torch.equal(g, G.gmm_logprobs_backward(Z, ids, r.lse, dlogp=w, stream=side))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc = G.gmm_logprobs(Z, ids, m=4)
        gc = G.gmm_logprobs_backward(Z, ids, rc.lse, dlogp=w)
    for _ in range(2):
        Z.normal_()
        graph.replay()
        want = G.gmm_logprobs(Z, ids, m=4)
        for u, v in zip(rc, want):
            assert torch.equal(u, v)
        assert torch.equal(gc, G.gmm_logprobs_backward(Z, ids, want.lse, dlogp=w))


def test_no_rows(G):
    import torch

    Z = torch.empty(0, 100, device="cuda")
    r = G.gmm_logprobs(Z, torch.empty(0, dtype=torch.int32, device="cuda"), m=3)
    assert r.lse.shape == (0,) and r.top_idx.shape == (0, 3)
    assert G.gmm_logprobs_backward(Z, None, r.lse, dlse=r.lse).shape == (0, 100)
    assert G.gmm_route(Z, 2)[0].shape == (0, 2)
