"""gmm_beam_select and gmm_beam_reorder on the GPU against oracle/assignments.py, and a decode and a
training step that use the operators around a vocabulary and a router together.

A score is off by the error of the row's first log p, which test_posteriors_gpu.py derives (s + 4 u
(2 |z| + |log p|) with u = 2^-24 and s = u (2 |z| + 387 + K / 256)), and by its rounding to float32,
u |score|.  A candidate may take the place of another whose score is no further off than twice that.
"""
import numpy as np
import pytest

from oracle import assignments as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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


def _logits(rng, N, K, dtype, pad=0, shift=0, masks=False):
    import torch

    x = (rng.normal(size=(N, K)) * 2.5).astype(np.float32)
    x[np.arange(N), rng.integers(0, K, N)] += 6
    if masks:
        x[rng.random((N, K)) < 0.3] = -np.inf
        x[::5] = -np.inf
        x[1::7] = np.finfo(np.float16).min if dtype == "f16" else -3e38
    buf = torch.full((N * (K + pad) + shift + 64,), float("nan"), dtype=_t(dtype), device="cuda")
    Z = buf[shift:shift + N * (K + pad)].view(N, K + pad)[:, :K]
    Z.copy_(torch.from_numpy(x))
    return Z, Z.float().cpu().numpy()


def _check(r, x, scores, m, ended=None, end_id=0, scale=1.0):
    B, w = scores.shape
    K = x.shape[1]
    want = A.beam_select(x, scores, m, ended, end_id, scale)
    q = A.beam_scores(x, scores, ended, end_id, scale)
    s, p, t = (v.cpu().numpy() for v in r)
    big = np.abs(np.where(np.isfinite(x) & (np.abs(x) < 1e4), x, 0)).max() * scale
    for b in range(B):
        np.testing.assert_array_equal(p[b] < 0, want[1][b] < 0)
        np.testing.assert_array_equal(t[b] < 0, want[2][b] < 0)
        n = int((p[b] >= 0).sum())
        assert (s[b, n:] == -np.inf).all() and len(set(zip(p[b, :n], t[b, :n]))) == n
        true = q[b, p[b, :n], t[b, :n]]
        top = np.where(np.isfinite(want[0][b, :n]), np.abs(want[0][b, :n]), 0)
        tol = U * (2 * big + 387 + K / 256) + 4 * U * (2 * big + top) + U * top
        with np.errstate(over="ignore"):
            near = np.abs(np.where(s[b, :n] == np.float32(true), 0, s[b, :n] - true))
        assert (near <= tol).all()
        assert (np.abs(true - want[0][b, :n]) <= 2 * tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,w,K,m,pad,shift,masks", [
    (1, 1, 1, 1, 0, 0, False), (1, 1, 9, 4, 0, 0, False), (2, 3, 5, 20, 0, 1, True),
    (3, 4, 300, 8, 8, 0, True), (5, 8, 1000, 16, 3, 2, False), (2, 32, 1025, 32, 0, 0, True),
    (9, 2, 5000, 2, 0, 0, True), (1, 5, 33_333, 10, 1, 0, False), (40, 7, 129, 7, 0, 0, True),
])
def test_selection(G, B, w, K, m, pad, shift, masks, dtype):
    import torch

    rng = np.random.default_rng(K + w)
    Z, x = _logits(rng, B * w, K, dtype, pad, shift, masks)
    scores = rng.normal(size=(B, w)).astype(np.float32) * 3 - 20
    ended = None
    if masks:
        ended = rng.random((B, w)) < 0.2
        scores[rng.random((B, w)) < 0.2] = -np.inf
    r = G.gmm_beam_select(Z, torch.from_numpy(scores).cuda(), m,
                          None if ended is None else torch.from_numpy(ended).cuda(), K // 2, 0.75)
    _check(r, x, scores, m, ended, K // 2, 0.75)


def test_equal_scores_go_to_the_lower_beam_then_logit_then_class(G):
    import torch

    Z = torch.full((4, 16), -float("inf"), device="cuda")
    Z[:, [3, 9]] = 1.0
    Z[2, 5] = 1.0
    Z[3, 3] = -float("inf")
    s = torch.tensor([[0.0, 0.0], [0.0, 0.0]], device="cuda")
    r = G.gmm_beam_select(Z, s, 4)
    assert r.parent.tolist() == [[0, 0, 1, 1], [1, 0, 0, 0]]
    assert r.token.tolist() == [[3, 9, 3, 9], [9, 3, 5, 9]]
    assert r.scores[1, 0].item() == 0.0
    ended = torch.tensor([[1, 1], [0, 1]], dtype=torch.uint8, device="cuda")
    r = G.gmm_beam_select(Z, s, 3, ended=ended, end_id=7)
    assert r.parent.tolist() == [[0, 1, -1], [1, 0, 0]]
    assert r.token.tolist() == [[7, 7, -1], [7, 3, 5]]


def test_scores_that_float32_cannot_tell_apart(G):
    """Two beams 3e-7 apart at scores of -20, where float32 steps by 1.9e-6: the classes decide.
    (The logits are powers of 2 times small whole numbers, so both rows' sums are alike.)"""
    import torch

    K = 64
    Z = torch.zeros(2, K, device="cuda")
    Z[0, 10], Z[1, 40] = 2.0, 2.0 + 2.0 ** -20
    s = torch.full((1, 2), -20.0, device="cuda")
    r = G.gmm_beam_select(Z, s, 2)
    assert r.parent.tolist() == [[1, 0]] and r.token.tolist() == [[40, 10]]
    assert abs(r.scores[0, 0].item() - r.scores[0, 1].item()) <= 4e-6


def test_logits_whose_products_with_the_scale_are_equal(G):
    """Two neighbours among the float32 numbers whose products with 0.75 round to one: in the order
    of gmm_logprobs they are equal, but the larger one's score is 1.4e-6 higher.  Each beam offers
    its m best classes in that order; candidates are put in the order of their scores."""
    import torch

    f = np.float32
    small = next(x for x in np.arange(f(22), f(23), f(2) ** -19, dtype=f)
                 if x * f(0.75) == (x + f(2) ** -19) * f(0.75))
    large = small + f(2) ** -19
    Z = torch.full((2, 16), -float("inf"), device="cuda")
    Z[0, 3], Z[0, 9], Z[1, 3], Z[1, 9] = map(float, (small, large, large, small))
    s = torch.tensor([[0.0, -7e-7]], device="cuda")
    want = A.beam_select(Z.cpu().numpy(), s.cpu().numpy(), 4, scale=0.75)
    assert want[1].tolist() == [[0, 1, 0, 1]] and want[2].tolist() == [[9, 3, 3, 9]]
    for m in (2, 3, 4):
        r = G.gmm_beam_select(Z, s, m, scale=0.75)
        assert r.parent.tolist() == want[1][:, :m].tolist()
        assert r.token.tolist() == want[2][:, :m].tolist()
        assert (r.scores[0].double().cpu() - torch.from_numpy(want[0][0, :m])).abs().max() < 2e-7
    one = G.gmm_beam_select(Z[:1], s[:, :1], 2, scale=0.75)
    assert one.token.tolist() == [[9, 3]] and one.scores[0, 0] > one.scores[0, 1]
    one = G.gmm_beam_select(Z[:1], s[:, :1], 1, scale=0.75)
    assert one.token.tolist() == G.gmm_logprobs(Z[:1], m=1, scale=0.75).top_idx.tolist() == [[3]]


@pytest.mark.parametrize("B,w,K,m", [(3, 1, 40, 8), (5, 4, 300, 32), (2, 32, 70, 32), (4, 3, 5000, 9)])
def test_candidates_of_a_beam_follow_their_logits(G, B, w, K, m):
    """Logits a few float32 steps apart, at a scale that makes many products equal."""
    import torch

    rng = np.random.default_rng(K + m)
    x = (22 + rng.integers(0, 12, (B * w, K)) * 2.0 ** -19).astype(np.float32)
    z = x * np.float32(0.75)
    s = (rng.integers(0, 3, (B, w)) * 1e-6).astype(np.float32)
    r = G.gmm_beam_select(torch.from_numpy(x).cuda(), torch.from_numpy(s).cuda(), m, scale=0.75)
    scores, parent, token = (t.cpu().numpy() for t in r)
    assert (np.diff(scores, axis=1) <= 0).all() and (parent >= 0).all()
    for b in range(B):
        for i in range(w):
            row = b * w + i
            taken = token[b, parent[b] == i]
            best = np.lexsort((np.arange(K), -z[row]))[:m]  # what the beam offers
            best = best[np.lexsort((np.arange(len(best)), -x[row, best].astype(np.float64)))]
            np.testing.assert_array_equal(taken, best[:len(taken)])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,spread", [(50, 1.0), (1000, 0.1), (5000, 1.0), (131_072, 0.1)])
def test_beams_of_flat_rows(G, K, spread, dtype):
    """The best candidates of two beams 2.2 times the bound of a log p apart: in the order that 64
    bits give them."""
    import torch

    B = 24
    rng = np.random.default_rng(K)
    Z = torch.from_numpy((rng.normal(size=(2 * B, K)) * spread).astype(np.float32)).to(_t(dtype))
    x = Z.float().numpy()
    best = A.beam_scores(x, np.zeros((B, 2), np.float32), scale=0.75).max(2)
    big = 0.75 * np.abs(x).max()
    bound = U * (2 * big + 387 + K / 256) + 4 * U * (2 * big + np.abs(best).max())
    sign = np.where(rng.random(B) < 0.5, -1.0, 1.0)
    scores = np.stack([np.zeros(B), best[:, 0] - best[:, 1] + 2.2 * sign * bound], 1)
    scores = scores.astype(np.float32)
    r = G.gmm_beam_select(Z.cuda(), torch.from_numpy(scores).cuda(), 2, scale=0.75)
    np.testing.assert_array_equal(r.parent[:, 0].cpu().numpy(), sign > 0)
    off = np.abs(r.scores[:, 0].double().cpu().numpy() - (best + scores.astype(np.float64)).max(1))
    assert (off <= bound + U * (np.abs(best).max() + 1)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("K", [100, 3000])
def test_what_is_not_a_number(G, K, bad):
    import torch

    rng = np.random.default_rng(2)
    Z, x = _logits(rng, 8, K, "f32")
    s = torch.zeros(4, 2, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = G.gmm_beam_select(Z, s, dev_flags=flags)
    s[1, 1] = -float("inf")
    Z[3, 5] = bad  # of a beam that is none
    ended = torch.zeros(4, 2, dtype=torch.bool, device="cuda")
    ended[3, 0] = True
    Z[6, 7] = bad  # of a beam that has ended
    r = G.gmm_beam_select(Z, s, ended=ended, dev_flags=flags)
    assert flags.item() == 0 and r.scores.isfinite().all()
    assert torch.equal(r.token[[0, 2]], want.token[[0, 2]])
    Z[4, K - 1] = bad
    r = G.gmm_beam_select(Z, s, ended=ended, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_NONFINITE_X
    assert r.scores[2].isnan().all() and (r.parent[2] == -1).all() and (r.token[2] == -1).all()
    assert torch.equal(r.token[0], want.token[0]) and r.scores[[0, 1, 3]].isfinite().all()
    flags.zero_()
    s[0, 0] = bad
    r = G.gmm_beam_select(Z, s, ended=ended, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_NONFINITE_X and r.scores[0].isnan().all()


def test_no_beams(G):
    import torch

    r = G.gmm_beam_select(torch.zeros(0, 9, device="cuda"), torch.zeros(0, 3, device="cuda"))
    assert r.scores.shape == (0, 3)
    r = G.gmm_beam_select(torch.zeros(2, 9, device="cuda"),
                          torch.full((1, 2), -float("inf"), device="cuda"))
    assert (r.scores == -float("inf")).all() and (r.parent == -1).all()
    t = torch.ones(2, 3, device="cuda")
    G.gmm_beam_reorder([], torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    G.gmm_beam_reorder(t[:0], torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    G.gmm_beam_reorder(t[:, :0], torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    assert (t == 1).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "uint8", "int64"])
@pytest.mark.parametrize("B,w,shape,dim,lens", [
    (1, 2, (3,), None, False), (3, 4, (2, 17, 24), 2, True), (5, 8, (17, 3), 1, True),
    (2, 32, (3, 50, 8), 2, True), (7, 1, (4, 4), 1, False), (1500, 3, (2, 5, 16), 2, True),
    (2, 5, (40, 16), 1, True), (4, 16, (1, 9, 1), 2, True), (2, 9, (3, 2, 11, 33), 3, True),
])
def test_states_follow_their_parents(G, B, w, shape, dim, lens, dtype):
    import torch

    rng = np.random.default_rng(B + w)
    t = torch.from_numpy(rng.integers(0, 250, (B * w,) + shape)).to(getattr(torch, dtype)).cuda()
    parent = rng.integers(-1, w, (B, w)).astype(np.int32)
    if B > 2:
        parent[1] = np.arange(w)  # a group that stays
    n = rng.integers(0, shape[dim - 1] + 1, B).astype(np.int32) if lens else None
    want = A.beam_reorder(t.float().cpu().numpy(), parent, n, dim)
    G.gmm_beam_reorder(t, torch.from_numpy(parent).cuda(),
                       None if n is None else torch.from_numpy(n).cuda(), dim)
    np.testing.assert_array_equal(t.float().cpu().numpy(), want)


def test_many_states_of_all_kinds(G):
    """More than one launch holds, mixed alignments, rows inside other tensors, with and without
    positions; what lies between stays as it is."""
    import torch

    rng = np.random.default_rng(4)
    B, w = 3, 4
    parent = rng.integers(0, w, (B, w)).astype(np.int32)
    lens = np.array([0, 5, 9], np.int32)
    states, dims = [], []
    layers = torch.randn(35, B * w, 2, 9, 8, device="cuda")
    for i in range(35):
        states.append(layers[i])
        dims.append(2)
    history = torch.randint(0, 99, (B * w, 12), device="cuda", dtype=torch.int32)
    states += [history[:, :9], torch.randn(B * w, 5, device="cuda").half(),
               torch.randn(B * w, 9, 3, device="cuda").half()]
    dims += [1, None, 1]
    behind = history[:, 9:].clone()
    want = [A.beam_reorder(t.double().cpu().numpy(), parent, lens, d)
            for t, d in zip(states, dims)]
    G.gmm_beam_reorder(states, torch.from_numpy(parent).cuda(), torch.from_numpy(lens).cuda(), dims)
    for t, v in zip(states, want):
        np.testing.assert_array_equal(t.double().cpu().numpy(), v)
    assert torch.equal(history[:, 9:], behind)


def test_bad_parents_and_lengths_are_told(G):
    import torch

    t = torch.arange(8, device="cuda", dtype=torch.float32).view(4, 2)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    parent = torch.tensor([[1, -1], [0, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    G.gmm_beam_reorder(t, parent, lens, 1, dev_flags=flags)
    assert flags.item() == 0 and t.tolist() == [[2, 1], [2, 3], [4, 5], [4, 5]]
    parent[0, 1], parent[0, 0] = 2, 0
    G.gmm_beam_reorder(t, parent, lens, 1, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    assert t.tolist() == [[2, 1], [2, 3], [4, 5], [4, 5]]
    flags.zero_()
    parent.copy_(torch.tensor([[1, 0], [0, 1]]))
    lens.copy_(torch.tensor([3, 2]))
    G.gmm_beam_reorder(t, parent, lens, 1, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    assert t.tolist() == [[2, 3], [2, 1], [4, 5], [4, 5]]


def test_a_state_beyond_32_bits(G):
    import torch

    t = torch.zeros(4, 3, 400_000, 512, dtype=torch.bfloat16, device="cuda")  # 1.2 GB a row
    t[:, :, 399_990:, :] = torch.randn(4, 3, 10, 512, device="cuda").bfloat16()
    tail = t[:, :, 399_990:].clone()
    parent = torch.tensor([[3, 1], [1, 1]], dtype=torch.int32, device="cuda")
    G.gmm_beam_reorder(t, parent, None, 2)  # (3 is no beam of the group)
    assert torch.equal(t[0, :, 399_990:], tail[0]) and torch.equal(t[2, :, 399_990:], tail[3])
    assert t[2].count_nonzero() == tail[3].count_nonzero()
    t[2].zero_()
    G.gmm_beam_reorder(t, parent, torch.tensor([0, 399_995], dtype=torch.int32, device="cuda"), 2)
    assert torch.equal(t[2, :, 399_990:399_995], tail[3, :, :5])
    assert t[2, :, 399_995:].count_nonzero() == 0


def test_captured_and_on_another_stream(G):
    import torch

    rng = np.random.default_rng(5)
    Z, _ = _logits(rng, 12, 2000, "bf16")
    s = torch.randn(3, 4, device="cuda")
    want = G.gmm_beam_select(Z, s, 4)
    cache = torch.randn(12, 2, 30, 16, device="cuda")
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    a = cache.clone()
    torch.cuda.synchronize()
    r = G.gmm_beam_select(Z, s, 4, stream=other)
    G.gmm_beam_reorder(a, r.parent, None, 2, stream=other)
    other.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(r, want))
    b = cache.clone()
    ws = torch.empty(G.gmm_beam_workspace_size(Z, 4, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = G.gmm_beam_select(Z, s, 4, ws=ws)
        G.gmm_beam_reorder(b, r.parent, None, 2)
    b.copy_(cache)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(p, q) for p, q in zip(r, want))
    Z.neg_()
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(r, G.gmm_beam_select(Z, s, 4)))


def test_two_threads_on_two_streams(G):
    """Calls at the same time, each with memory of its own, give what they give alone."""
    import threading

    import torch

    def work(seed, stream):
        rng = np.random.default_rng(seed)
        with torch.cuda.stream(stream):
            Z, _ = _logits(rng, 24, 3000, "bf16")
            s = torch.from_numpy(rng.normal(size=(6, 4)).astype(np.float32)).cuda()
            W = torch.from_numpy(rng.normal(size=(4000, 64)).astype(np.float32)).cuda()
            ids = torch.from_numpy(rng.integers(0, 4000, 5000).astype(np.int32)).cuda()
            cache = torch.from_numpy(rng.normal(size=(24, 2, 40, 16)).astype(np.float32)).cuda()
            results = []
            for _ in range(30):
                r = G.gmm_beam_select(Z, s)
                c = cache.clone()
                G.gmm_beam_reorder(c, r.parent, None, 2)
                x = G.gmm_embed(W, ids)
                dW, _ = G.gmm_embed_backward(x, ids, 4000)
                idx, _ = G.gmm_route(x, 4)
                loss = G.gmm_route_loss(x, idx)
                results.append((*r, c, x, dW, *loss))
            stream.synchronize()
        return results

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone = [work(i, streams[i])[0] for i in range(2)]
    together = [None, None]
    threads = [threading.Thread(target=lambda i=i: together.__setitem__(i, work(i, streams[i])))
               for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for want, got in zip(alone, together):
        for r in got:
            assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_refusals(G):
    import torch

    Z, s = torch.zeros(6, 8, device="cuda"), torch.zeros(2, 3, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for bad in (lambda: G.gmm_beam_select(Z, s[0]), lambda: G.gmm_beam_select(Z, s.double()),
                lambda: G.gmm_beam_select(Z[:5], s), lambda: G.gmm_beam_select(Z, s.cpu()),
                lambda: G.gmm_beam_select(Z, s.t()),
                lambda: G.gmm_beam_select(Z, s, ended=s),
                lambda: G.gmm_beam_select(Z, s, ended=torch.zeros(6, dtype=torch.bool,
                                                                  device="cuda")),
                lambda: G.gmm_beam_reorder(Z[:5], p), lambda: G.gmm_beam_reorder(Z, p.long()),
                lambda: G.gmm_beam_reorder(Z, p, dim=0), lambda: G.gmm_beam_reorder(Z, p, dim=2),
                lambda: G.gmm_beam_reorder([Z, Z], p, dim=[1]),
                lambda: G.gmm_beam_reorder(Z.cpu(), p), lambda: G.gmm_beam_reorder(Z, p.t()),
                lambda: G.gmm_beam_reorder(Z[:, ::2], p),
                lambda: G.gmm_beam_reorder(Z, p, lens=p[0])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: G.gmm_beam_select(Z, s, 33), lambda: G.gmm_beam_select(Z, s, 0),
                lambda: G.gmm_beam_select(Z, s, ended=torch.zeros(2, 3, dtype=torch.bool,
                                                                  device="cuda"), end_id=8),
                lambda: G.gmm_beam_select(torch.zeros(33, 8, device="cuda"),
                                          torch.zeros(1, 33, device="cuda")),
                lambda: G.gmm_beam_select(Z, s, scale=0.0),
                lambda: G.gmm_beam_select(Z, s, ws=torch.zeros(256, dtype=torch.uint8,
                                                               device="cuda")),
                lambda: G.gmm_beam_reorder(Z[:1].expand(6, 8), p)):
        with pytest.raises(G.GmmError):
            bad()


def test_a_small_model_decodes_with_beams(G):
    """Tokens are embedded, routed and run through experts, their state summed along the way, and
    the head's logits continued by beams whose states follow: as the same in plain steps finds."""
    import torch

    torch.manual_seed(0)
    V, D, E, F, m, B, w, steps = 500, 64, 8, 32, 2, 2, 3, 5
    bf = dict(dtype=torch.bfloat16, device="cuda")
    W = torch.randn(V, D, **bf)
    head, router = torch.randn(V, D, **bf) / 4, torch.randn(E, D, **bf) / 4
    up, down = torch.randn(E, 2 * F, D, **bf) / 8, torch.randn(E, D, F, **bf) / 6
    token = torch.tensor([[3, -1, -1], [7, -1, -1]], dtype=torch.int32, device="cuda")
    scores = torch.tensor([[0.0, -np.inf, -np.inf]] * B, device="cuda")
    state = torch.zeros(B * w, D, **bf)
    history = torch.zeros(B * w, steps, dtype=torch.int32, device="cuda")
    used = torch.zeros(B, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(steps):
        x = G.gmm_embed(W, token.view(-1), scale=0.5, dev_flags=flags)
        idx, resp = G.gmm_route(x @ router.T, m, renorm=True)
        state += G.gmm_moe(x, idx, resp, up, down)
        logits = state @ head.T
        r = G.gmm_beam_select(logits, scores, dev_flags=flags)
        _check(r, logits.float().cpu().numpy(), scores.cpu().numpy(), w)
        before, past = state.clone(), history.clone()
        G.gmm_beam_reorder([state, history], r.parent, used, [None, 1], dev_flags=flags)
        rows = (r.parent + torch.arange(B, device="cuda")[:, None] * w).view(-1).long()
        assert torch.equal(state, before[rows]) and torch.equal(history[:, :t], past[rows][:, :t])
        token, scores = r.token, r.scores
        history[:, t] = token.view(-1)
        used += 1
        assert (token >= 0).all() and (token < V).all()
    assert flags.item() == 0
    assert len({tuple(h) for h in history.tolist()}) == B * w  # no two beams are the same


def test_a_training_step_of_embedding_and_router(G):
    """y = sum_j resp_j x_n C[idx_j] over the routed entries of a small table, a loss on y, on the
    balance and on z: all gradients against torch's autograd in 64 bits, counts held fixed."""
    import torch

    torch.manual_seed(1)
    N, V, D, E, m = 200, 90, 32, 12, 3
    W = torch.randn(V, D, device="cuda")
    R, C = torch.randn(E, D, device="cuda") / 3, torch.randn(E, D, device="cuda")
    ids = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    ids[::13] = -1
    target = torch.randn(N, D, device="cuda")
    x = G.gmm_embed(W, ids, scale=0.7)
    logits = x @ R.T
    idx, resp = G.gmm_route(logits, m, renorm=True)
    mask = ids >= 0
    loss = G.gmm_route_loss(logits, idx, mask=mask)
    y = G.gmm_embed(C, idx, resp)
    dy = (y - target) / N
    dC, dresp = G.gmm_embed_backward(dy, idx, E, resp, W=C)
    coef = torch.tensor([0.01], device="cuda"), torch.tensor([0.001], device="cuda")
    dlogits = G.gmm_route_backward(logits, idx, dresp, True, loss.counts, loss.rows, *coef,
                                   mask=mask)
    dR, dx = dlogits.T @ x, dlogits @ R
    dW, _ = G.gmm_embed_backward(dx, ids, V, scale=0.7)

    W6, R6, C6 = (t.double().requires_grad_() for t in (W, R, C))
    live = mask.double()[:, None]
    x6 = 0.7 * W6[ids.clamp(min=0).long()] * live
    l6 = x6 @ R6.T
    p = torch.softmax(l6, 1)
    q = p.gather(1, idx.long())
    q = q / q.sum(1, keepdim=True)
    y6 = (q[:, :, None] * C6[idx.long()]).sum(1)
    L = mask.sum()
    f = loss.counts[0].double() / (m * L)
    value = ((y6 - target.double()) ** 2).sum() / (2 * N)
    value = value + 0.01 * E * (f * (p * live).sum(0) / L).sum()
    value = value + 0.001 * (torch.logsumexp(l6, 1) ** 2 * live[:, 0]).sum() / L
    want = torch.autograd.grad(value, (W6, R6, C6))
    assert abs(loss.balance.item() - (E * (f * (p * live).sum(0) / L).sum()).item()) < 1e-5
    for got, exact in zip((dW, dR, dC), want):
        # sums of up to 200 float32 products, three in a row: 600 u of the largest, doubled
        assert (got.double() - exact).abs().max() < 1200 * U * exact.abs().max() + 1e-7
