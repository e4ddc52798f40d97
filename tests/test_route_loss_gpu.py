"""gmm_route_loss and gmm_route_backward on the GPU against oracle/assignments.py.

Tolerances, for u = 2^-24.  An exponent d = scale (x - largest x) is off by 3 u |d| (difference,
product, the constant log2 e), the hardware exponential by 2^-22 in relation, and e^d is 0 where
d < -104: so e^d, their sum S (K / 8 terms a lane and 5 levels) and p = e^d / S are off by at most
  s = 2 (3 * 104 u + 4 u) + (K / 8 + 10) u  in relation.
load adds sums over a thread's rows (at most N / 8 of a CTA's, and 12 joining steps; then 64 bits):
s + (N / 8 + 14) u; balance the same.  lse is off by s / 2 + 2 u (|largest z| + |lse|), lse^2 by
twice |lse| times that, and its sum by (N / 8 + 14) u in relation.
Gradient: every product of the formula by 2 s + (K / 8 + 30) u times its terms' magnitudes (lse's
own error is below s (1 + |lse|)), then half a step of the type, and half its smallest step.
"""
import numpy as np
import pytest

from oracle import assignments as A
from oracle import posteriors as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


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


def _s(K):
    return 2 * (3 * 104 * U + 4 * U) + (K / 8 + 10) * U


def _case(seed, N, K, m, dtype, S=0, masks=False, pad=0, shift=0, spread=2.0):
    """Logits (in rows of K + pad, `shift` entries into NaN), choices, mask and offsets."""
    import torch

    rng = np.random.default_rng(seed)
    x = (rng.normal(size=(N, K)) * spread).astype(np.float32)
    if masks and N:
        x[rng.random((N, K)) < 0.2] = -np.inf
        x[rng.integers(0, N, N // 20 + 1)] = -np.inf  # rows with nothing left
        low = np.finfo(np.float16).min if dtype == "f16" else -3e38
        x[0, K // 2:] = low
    buf = torch.full((N * (K + pad) + shift + 64,), float("nan"), dtype=_t(dtype), device="cuda")
    Z = buf[shift:shift + N * (K + pad)].view(N, K + pad)[:, :K]
    Z.copy_(torch.from_numpy(x))
    x = Z.float().cpu().numpy()
    idx = P.order(x.astype(np.float64), m)
    if N > 2 and masks:
        idx[1, :] = -1
    mask = rng.random(N) < 0.8 if masks else None
    offsets = None
    if S:
        offsets = np.sort(rng.integers(0, N + 1, S + 1)).astype(np.int32)
        if S > 3:
            offsets[2] = offsets[1]  # an empty segment
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    return Z, x, idx, mask, offsets, cuda(idx), cuda(mask), cuda(offsets), rng


CASES = [  # N, K, m, S, masks, pad, shift
    (1, 1, 1, 0, False, 0, 0), (1, 8, 2, 0, False, 0, 0), (7, 5, 3, 3, True, 0, 1),
    (100, 64, 8, 0, False, 0, 0), (333, 65, 4, 5, True, 3, 0), (1000, 128, 6, 40, True, 8, 0),
    (2500, 256, 8, 7, True, 0, 0), (513, 300, 2, 2, False, 4, 3), (700, 512, 8, 0, True, 0, 0),
    (400, 1024, 1, 300, True, 0, 0), (64, 1023, 8, 1, True, 0, 0), (12_000, 16, 2, 900, True, 0, 0),
    (20_000, 33, 8, 0, False, 0, 0), (5, 3, 8, 1, True, 0, 0),
    # beside the numbers of rows at which one launch becomes two
    (256, 64, 2, 3, True, 0, 0), (257, 64, 2, 3, True, 0, 0), (128, 256, 2, 0, True, 0, 0),
    (129, 256, 2, 0, True, 0, 0), (64, 600, 2, 2, True, 0, 0), (65, 600, 2, 2, True, 0, 0),
    (200, 7, 2, 500, True, 0, 0),
    # several CTAs to a segment, whole shares and not, and where there are too many rows for that
    (63, 64, 2, 0, True, 0, 0), (191, 64, 2, 0, True, 3, 0), (1536, 64, 2, 0, True, 0, 0),
    (1537, 64, 2, 0, True, 0, 0), (2047, 40, 3, 5, True, 0, 1), (2049, 40, 3, 5, True, 0, 0),
    (768, 250, 2, 0, True, 0, 0), (769, 250, 2, 1, True, 0, 0), (384, 600, 2, 0, True, 0, 0),
    (385, 600, 2, 2, True, 0, 0), (512, 64, 2, 100, True, 0, 0), (513, 64, 2, 100, True, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K,m,S,masks,pad,shift", CASES)
def test_losses(G, N, K, m, S, masks, pad, shift, dtype):
    Z, x, i, mask, off, idx, dmask, doff, _ = _case(N + K, N, K, m, dtype, S, masks, pad, shift)
    got = G.gmm_route_loss(Z, idx, offsets=doff, mask=dmask, scale=0.75)
    balance, z, load, counts, rows = A.route_loss(x, i, off, mask, 0.75)
    np.testing.assert_array_equal(got.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(got.rows.cpu().numpy(), rows)
    tol = _s(K) + (N / 8 + 14) * U
    for name, want in (("load", load), ("balance", balance)):
        have = getattr(got, name).double().cpu().numpy()
        assert (np.abs(have - want) <= tol * np.abs(want) + 1e-40).all(), name
    ordinary = np.where(np.isfinite(x) & (x > -1e4), x, 0)
    size = 0.75 * np.abs(ordinary).max() + np.log(K) + 1
    have = got.z.double().cpu().numpy()
    # a row of nothing but -3e38 has lse = -2.25e38: its square divided by fewer than 2^20 rows is
    # above 2^128, which float32 rounds to infinity
    over = z >= 2.0 ** 128
    assert (have[over] == np.inf).all()
    have, z = have[~over], z[~over]
    assert (np.abs(have - z) <= 2 * size * (_s(K) / 2 + 4 * U * size) + (N / 8 + 14) * U * z).all()
    again = G.gmm_route_loss(Z, idx, offsets=doff, mask=dmask, scale=0.75)
    for a, b in zip(got, again):
        assert (a == b).all()


@pytest.mark.parametrize("what,renorm,dtype", [
    (what, renorm, dtype)
    for what, kinds, types in (("all", (0, 1), ("f32", "bf16", "f16")),
                               ("weights", (0, 1), ("f32", "bf16")),
                               ("balance", (0,), ("f32", "bf16")), ("z", (0,), ("f32", "bf16")))
    for renorm in kinds for dtype in types])
@pytest.mark.parametrize("N,K,m,S,masks,pad,shift", CASES)
def test_gradient(G, N, K, m, S, masks, pad, shift, dtype, renorm, what):
    import torch

    renorm = bool(renorm)
    Z, x, i, mask, off, idx, dmask, doff, rng = _case(N + K + 1, N, K, m, dtype, S, masks, pad,
                                                      shift)
    S = max(S, 1)
    _, _, _, counts, rows = A.route_loss(x, i, off, mask, 0.75)
    up = dict(dresp=rng.normal(size=(N, m)) if what in ("all", "weights") else None,
              dbalance=rng.normal(size=S) * N if what in ("all", "balance") else None,
              dz=rng.normal(size=S) * N if what in ("all", "z") else None)
    up = {k: None if v is None else v.astype(np.float32) for k, v in up.items()}
    dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in up.items()}
    got = G.gmm_route_backward(Z, idx, dev["dresp"], renorm,
                               torch.from_numpy(counts.astype(np.int32)).cuda(),
                               torch.from_numpy(rows.astype(np.int32)).cuda(), dev["dbalance"],
                               dev["dz"], doff, dmask, 0.75)
    want, size = A.route_backward(x, i, up["dresp"], renorm, counts, rows, up["dbalance"],
                                  up["dz"], off, mask, 0.75)
    top = np.abs(np.where(np.isfinite(x) & (x > -1e4), x, 0)).max()
    tol = (2 * _s(K) + (K / 8 + 30) * U + 8 * U * top) * size
    if up["dz"] is not None:  # lse's own error, times 2 |dz| / L of the row's segment
        o = [0, N] if off is None else off
        for seg in range(S):
            tol[o[seg]:o[seg + 1]] += 0.75 * 2 * abs(up["dz"][seg]) / max(1, rows[seg]) * (
                _s(K) + 4 * U * (top + np.log(K) + 1))
    tol = tol + HALF[dtype] * np.abs(want) + LEAST[dtype]
    have = got.double().cpu().numpy()
    # beyond float16's largest value (65504, and half a step of 32) a result is infinite: a segment
    # of one row has gradients of up to N K
    if dtype == "f16":
        over = np.abs(want) > 65520
        assert (np.isinf(have) | ~over | (np.abs(want) - tol < 65520)).all()
        have = np.where(over, 0, have)
        want = np.where(over, 0, want)
    assert (np.abs(have - want) <= tol).all(), (np.abs(have - want) - tol).max()
    # in place, and from run to run
    flat = Z.clone() if pad == 0 else None
    if flat is not None:
        out = G.gmm_route_backward(flat, idx, dev["dresp"], renorm,
                                   torch.from_numpy(counts.astype(np.int32)).cuda(),
                                   torch.from_numpy(rows.astype(np.int32)).cuda(), dev["dbalance"],
                                   dev["dz"], doff, dmask, 0.75, out=flat)
        assert out is flat
        if shift == 0:
            assert torch.equal(flat, got)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("K", [3, 64, 250, 1000])
def test_an_expert_named_twice(G, K, renorm):
    """Choices that name the same expert: each counts, and its gradients add up."""
    import torch

    N, m = 60, 5
    Z, x, i, _, _, idx, _, _, rng = _case(K + 9, N, K, m, "f32")
    i[:, 1] = i[:, 0]
    i[::3, 4] = i[::3, 0]
    i[::4, 2:] = i[::4, 1:2]
    i[::7, 3] = -1
    i[5] = -1
    idx.copy_(torch.from_numpy(i))
    d = rng.normal(size=(N, m)).astype(np.float32)
    loss = G.gmm_route_loss(Z, idx)
    assert torch.equal(loss.counts[0].cpu(), torch.bincount(idx[idx >= 0].cpu(), minlength=K).int())
    got = G.gmm_route_backward(Z, idx, torch.from_numpy(d).cuda(), renorm).double().cpu().numpy()
    want, size = A.route_backward(x, i, d, renorm)
    top = np.abs(x).max()
    tol = (2 * _s(K) + (K / 8 + 30) * U + 8 * U * top) * size + HALF["f32"] * np.abs(want)
    assert (np.abs(got - want) <= tol + LEAST["f32"]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,pad,shift", [(64, 8, 0), (64, 3, 0), (200, 0, 1), (1000, 5, 3)])
def test_gradient_in_rows_of_another_tensor(G, K, pad, shift, dtype):
    """Rows of Z that start on 16 bytes and of dZ that do not: the same to a rounding of the type
    (vectors or single entries, the same arithmetic); what lies between the rows stays."""
    import torch

    N, m = 150, 4
    Z, x, i, _, _, idx, _, _, _ = _case(K, N, K, m, dtype)
    d, one = torch.randn(N, m, device="cuda"), torch.ones(1, device="cuda")
    loss = G.gmm_route_loss(Z, idx)
    args = (Z, idx, d, False, loss.counts, loss.rows, one, one)
    want = G.gmm_route_backward(*args).double()
    buf = torch.full((N * (K + pad) + shift + 64,), 7.0, dtype=_t(dtype), device="cuda")
    out = buf[shift:shift + N * (K + pad)].view(N, K + pad)[:, :K]
    assert G.gmm_route_backward(*args, out=out) is out
    # sums over lanes in another order: (K / 8 + 30) u of a row's largest terms, and a rounding
    tol = (K / 8 + 30) * U * 4 * want.abs().amax(1, keepdim=True) + 2 * HALF[dtype] * want.abs()
    assert ((out.double() - want).abs() <= tol + LEAST[dtype]).all()
    out.fill_(7.0)
    assert (buf == 7).all()


def test_gradient_is_what_the_losses_change_by(G):
    """Central differences of the library's own losses in float32: their error is that of the loss
    (a few 1e-7 of about 1) over the step, 1e-5 at a step of 0.05, plus the step's square times the
    third derivative, which is below 6 times the gradient's scale (2.5e-3 * 6 = 1.5e-2 of it)."""
    import torch

    N, K, m = 6, 5, 2
    Z, x, i, _, _, idx, _, _, _ = _case(5, N, K, m, "f32")
    base = G.gmm_route_loss(Z, idx)
    one = torch.ones(1, device="cuda")
    grad = G.gmm_route_backward(Z, idx, counts=base.counts, rows=base.rows, dbalance=one, dz=one)
    got = np.zeros((N, K))
    for n in range(N):
        for k in range(K):
            v = []
            for h in (0.05, -0.05):
                y = Z.clone()
                y[n, k] += h
                r = G.gmm_route_loss(y, idx)
                v.append((r.balance + r.z).item())
            got[n, k] = (v[0] - v[1]) / 0.1
    grad = grad.cpu().numpy()
    assert np.abs(got - grad).max() < 1e-4 + 1.5e-2 * np.abs(grad).max()


def test_a_sharded_batch_has_the_gradient_of_the_whole(G):
    """counts and rows summed over shards: each shard's rows get the whole batch's gradient."""
    import torch

    Z, x, i, _, _, idx, _, _, _ = _case(6, 200, 16, 2, "f32")
    whole = G.gmm_route_loss(Z, idx)
    one = torch.ones(1, device="cuda")
    want = G.gmm_route_backward(Z, idx, counts=whole.counts, rows=whole.rows, dbalance=one, dz=one)
    parts = [G.gmm_route_loss(Z[:70], idx[:70]), G.gmm_route_loss(Z[70:], idx[70:])]
    counts, rows = sum(p.counts for p in parts), sum(p.rows for p in parts)
    assert torch.equal(counts, whole.counts) and torch.equal(rows, whole.rows)
    got = torch.cat([G.gmm_route_backward(z, j, counts=counts, rows=rows, dbalance=one, dz=one)
                     for z, j in ((Z[:70], idx[:70]), (Z[70:], idx[70:]))])
    assert torch.equal(got, want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("K", [8, 200, 1000])
def test_what_is_not_a_number(G, K, bad):
    import torch

    Z, x, i, _, _, idx, _, _, _ = _case(7, 90, K, 2, "f32")
    off = torch.tensor([0, 30, 60, 80], dtype=torch.int32, device="cuda")
    mask = torch.ones(90, dtype=torch.bool, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    good = G.gmm_route_loss(Z, idx, off, mask, dev_flags=flags)
    want = G.gmm_route_backward(Z, idx, counts=good.counts, rows=good.rows, dbalance=one, dz=one,
                                offsets=off, mask=mask, dev_flags=flags)
    assert flags.item() == 0
    Z[85, 1] = bad  # in no segment
    mask[40] = False
    ref = G.gmm_route_loss(Z, idx, off, mask)
    Z[40, 1] = bad  # masked out
    r = G.gmm_route_loss(Z, idx, off, mask, dev_flags=flags)
    assert flags.item() == 0
    assert all(torch.equal(a, b) for a, b in zip(r, ref))
    g = G.gmm_route_backward(Z, idx, counts=r.counts, rows=r.rows, dbalance=one, dz=one,
                             offsets=off, mask=mask, dev_flags=flags)
    assert flags.item() == 0 and g.isfinite().all() and (g[[40, 85]] == 0).all()
    Z[45, K - 1] = bad
    r = G.gmm_route_loss(Z, idx, off, mask, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_NONFINITE_X
    assert r.balance.isnan().tolist() == [False, True, False]
    assert r.z.isnan().tolist() == [False, True, False]
    assert r.load[1].isnan().all() and r.load[[0, 2]].isfinite().all()
    flags.zero_()
    g = G.gmm_route_backward(Z, idx, counts=good.counts, rows=good.rows, dbalance=one, dz=one,
                             offsets=off, mask=mask, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_NONFINITE_X
    assert g[45].isnan().all() and g.isfinite().all(1).sum() == 89
    assert torch.equal(g[:30], want[:30])


def test_bad_indices_and_offsets_are_told(G):
    import torch

    Z, x, i, _, _, idx, _, _, _ = _case(8, 64, 16, 2, "f32")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = idx.clone()
    bad[3, 1], bad[9, 0] = 16, -2
    r = G.gmm_route_loss(Z, bad, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX and r.counts.sum() == 126
    flags.zero_()
    d = torch.ones(64, 2, device="cuda")
    g = G.gmm_route_backward(Z, bad, d, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    left = bad.clone()
    left[3, 1], left[9, 0] = -1, -1
    assert torch.equal(g, G.gmm_route_backward(Z, left, d))
    for off in ([0, 40, 30, 64], [0, 70], [-1, 64], [5, 2]):
        flags.zero_()
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        r = G.gmm_route_loss(Z, idx, offsets=o, dev_flags=flags)
        assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX, off
        assert r.balance.isnan().any()


def test_nothing_to_route(G):
    import torch

    Z = torch.zeros(0, 8, device="cuda")
    idx = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    r = G.gmm_route_loss(Z, idx)
    assert r.balance.item() == 0 and r.z.item() == 0 and r.rows.item() == 0
    assert (r.load == 0).all() and (r.counts == 0).all()
    assert G.gmm_route_backward(Z, idx, torch.zeros(0, 2, device="cuda")).shape == (0, 8)
    Z = torch.full((5, 8), -float("inf"), device="cuda")
    idx = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    r = G.gmm_route_loss(Z, idx)
    assert r.balance.item() == 0 and r.rows.item() == 0 and (r.load == 0).all()
    one = torch.ones(1, device="cuda")
    g = G.gmm_route_backward(Z, idx, torch.ones(5, 2, device="cuda"), True, r.counts, r.rows, one,
                             one)
    assert (g == 0).all()


@pytest.mark.parametrize("dtype,big,scale", [("f32", 1e38, 10.0), ("bf16", 1e38, 10.0),
                                             ("f16", 6e4, 1e34)])
@pytest.mark.parametrize("K", [8, 200, 1000])
@pytest.mark.parametrize("N", [90, 5000])  # one launch and two
def test_a_scaled_logit_that_overflows_is_masked_or_infinite(G, N, K, dtype, big, scale):
    """scale times a finite logit beyond float32's range: -inf is a masked class, +inf makes what
    the row is part of NaN, as in gmm_route's weights."""
    import torch

    spread = 0.0 if dtype == "f16" else 0.2
    Z, x, i, _, _, idx, _, _, rng = _case(8, N, K, 2, dtype, spread=spread)
    o = np.array([0, N // 3, 2 * N // 3, N - 10], np.int32)
    off, flags = torch.from_numpy(o).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    Z[N // 2 + 1, K // 2] = -big
    d = rng.normal(size=(N, 2)).astype(np.float32)
    dresp = torch.from_numpy(d).cuda()
    one = torch.ones(3, device="cuda")
    upstream = [dict(dresp=dresp), dict(dresp=dresp, renorm=True), dict(dbalance=one), dict(dz=one)]

    def loss():
        return G.gmm_route_loss(Z, idx, off, scale=scale, dev_flags=flags)

    def grad(r, kw):
        more = dict(counts=r.counts, rows=r.rows) if "dresp" not in kw else {}
        return G.gmm_route_backward(Z, idx, **kw, **more, offsets=off, scale=scale,
                                    dev_flags=flags)

    good = loss()
    want = [grad(good, kw) for kw in upstream]
    assert flags.item() == 0 and all(t.isfinite().all() for t in good)
    assert not any(t.isnan().any() for t in want)  # (1e34 times a probability: float16 has no room)
    b = N // 2
    Z[b, K - 1] = big
    x = Z.float().cpu().numpy()
    r = loss()
    assert flags.item() == G.GMM_DEVFLAG_NONFINITE_X
    for have, exact in zip(r[:3], A.route_loss(x, i, o, None, scale)):
        np.testing.assert_array_equal(have.isnan().cpu().numpy(), np.isnan(exact))
    assert r.balance.isnan().tolist() == r.z.isnan().tolist() == [False, True, False]
    assert r.load[1].isnan().all() and torch.equal(r.load[[0, 2]], good.load[[0, 2]])
    assert torch.equal(r.counts, good.counts) and torch.equal(r.rows, good.rows)
    assert G.gmm_route(Z, 2, scale=scale)[1][b].isnan().all()
    for kw, w in zip(upstream, want):
        flags.zero_()
        g = grad(good, kw)
        assert flags.item() == G.GMM_DEVFLAG_NONFINITE_X
        assert g[b].isnan().all(), kw.keys()
        g[b] = w[b]
        assert torch.equal(g, w)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("K", [8, 200, 1000])
def test_a_choice_that_the_scale_masks_has_no_weight(G, K, renorm):
    """A class is masked where its logit is -inf and where scale times its logit is."""
    import torch

    Z, x, i, _, _, _, _, _, rng = _case(10, 60, K, 3, "f32", spread=0.2)
    i[:, 1:] = [[1, 2]]
    i[::2, 0] = 0  # these rows name masked classes only
    i[1::2, 0] = 4
    Z[:, :3] = -1e38
    same = Z.clone()
    same[:, :3] = -np.inf
    idx = torch.from_numpy(i.astype(np.int32)).cuda()
    d = torch.from_numpy(rng.normal(size=(60, 3)).astype(np.float32)).cuda()
    got, want = [G.gmm_route_backward(z, idx, d, renorm, scale=10.0) for z in (Z, same)]
    assert torch.equal(got, want) and got.isfinite().all() and (got[::2] == 0).all()
    got, want = [G.gmm_route_loss(z, idx, scale=10.0) for z in (Z, same)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N,K,pad", [(1 << 28, 12, 4)])
def test_sums_over_many_like_rows(G, N, K, pad):
    """Logits of 0, as of a router that has not learnt: p = 1 / K and lse = log K in every row, and
    all roundings of a running sum go one way.  At most 512 of a lane's additions before 64 bits,
    and 14 to join lanes and warps; p is off by u, and log K by 2 u, its square by 5 u."""
    import torch

    Z = torch.zeros(N, K + pad, dtype=torch.bfloat16, device="cuda")[:, :K]
    idx = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    r = G.gmm_route_loss(Z, idx)
    assert r.rows.item() == N and r.counts[0].tolist() == [N] + [0] * (K - 1)
    assert (r.load.double() * K - 1).abs().max() <= (512 + 14 + 2) * U
    assert abs(r.balance.item() - 1) <= (512 + 14 + 2) * U
    assert abs(r.z.item() / np.log(K) ** 2 - 1) <= (512 + 14 + 6) * U


def test_captured_and_on_another_stream(G):
    import torch

    Z, x, i, _, off, idx, _, doff, _ = _case(9, 3000, 64, 4, "bf16", S=4)
    d = torch.randn(3000, 4, device="cuda")
    one = torch.ones(4, device="cuda")
    ws = torch.empty(G.gmm_route_loss_workspace_size(Z, 4), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    a = G.gmm_route_loss(Z, idx, doff, stream=other)
    b = G.gmm_route_backward(Z, idx, d, True, a.counts, a.rows, one, one, doff, stream=other)
    other.synchronize()
    r = G.gmm_route_loss(Z, idx, doff)
    assert all(torch.equal(p, q) for p, q in zip(a, r))
    assert torch.equal(b, G.gmm_route_backward(Z, idx, d, True, r.counts, r.rows, one, one, doff))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = G.gmm_route_loss(Z, idx, doff, ws=ws)
        g = G.gmm_route_backward(Z, idx, d, True, c.counts, c.rows, one, one, doff)
    for scale in (1.0, -0.5):
        Z.mul_(scale)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        r = G.gmm_route_loss(Z, idx, doff)
        assert all(torch.equal(p, q) for p, q in zip(c, r))
        assert torch.equal(g, G.gmm_route_backward(Z, idx, d, True, r.counts, r.rows, one, one,
                                                   doff))


def test_refusals(G):
    import torch

    Z = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    for bad in (lambda: G.gmm_route_loss(Z, idx.long()), lambda: G.gmm_route_loss(Z, idx[:3]),
                lambda: G.gmm_route_loss(Z, idx.cpu()), lambda: G.gmm_route_loss(Z.double(), idx),
                lambda: G.gmm_route_loss(Z, idx[0]),
                lambda: G.gmm_route_loss(Z, idx, mask=one),
                lambda: G.gmm_route_loss(Z, idx, offsets=one),
                lambda: G.gmm_route_backward(Z, idx, torch.zeros(4, 3, device="cuda")),
                lambda: G.gmm_route_backward(Z, idx, dbalance=one, counts=idx, rows=idx[0]),
                lambda: G.gmm_route_backward(Z, idx, torch.zeros(4, 2, device="cuda"),
                                             out=Z.half())):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: G.gmm_route_backward(Z, idx), lambda: G.gmm_route_backward(Z, idx, dz=one),
                lambda: G.gmm_route_loss(torch.zeros(4, 1025, device="cuda"), idx),
                lambda: G.gmm_route_loss(Z, torch.zeros(4, 9, dtype=torch.int32, device="cuda")),
                lambda: G.gmm_route_loss(Z, idx, ws=torch.zeros(64, dtype=torch.uint8,
                                                                device="cuda"))):
        with pytest.raises(G.GmmError):
            bad()
