"""gmm_moe on the GPU against oracle/posteriors.py.

Tolerance: the products of one output are summed in float32 by the tensor cores, 16 at a time,
over chains of at most n / 16 such steps (n = D or F), each step off by at most 2^-23 of the
magnitudes added so far; the inner activation is kept to 2^-17 or better in relation.  So an
element is off by at most (bound / |.| magnitudes) * ((D + F) / 16 + 64) 2^-23 + 2^-16 bound, and
half a step of the type on the whole.  `bound` is the oracle's sum of magnitudes.
"""
import numpy as np
import pytest

from oracle import posteriors as P
from soft_clustering_em_b200 import synth

pytestmark = pytest.mark.gpu


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

    return {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def _weights(rng, E, D, F, dtype):
    import torch

    out = []
    for shape, n in (((E, 2 * F, D), D), ((E, D, F), F)):
        w = (rng.normal(size=shape) / np.sqrt(n)).astype(np.float32)
        out.append(torch.from_numpy(w).to(_t(dtype)).cuda())
    return out


def _f64(*ts):
    return tuple(t.double().cpu().numpy() for t in ts)


def _check(G, X, idx, resp, W_up, W_down, act=0, out=None):
    import torch

    T, D = X.shape
    F = W_down.shape[2]
    p = G.moe_problem(X, idx, W_down, act, out)
    ws = torch.full((G.gmm_moe_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    Y = G.gmm_moe(X, idx, resp, W_up, W_down, act=act, out=out, ws=ws)
    rc, flags = G.gmm_device_status(ws)
    want, bound = P.moe(_f64(X)[0], idx.cpu().numpy(), _f64(resp)[0], *_f64(W_up, W_down), act)
    u = torch.finfo(X.dtype).eps / 2
    tol = (bound * (((D + F) / 16 + 64) * 2.0 ** -23 + 2.0 ** -16) + np.abs(want) * u
           + torch.finfo(X.dtype).smallest_normal * u)
    off = np.abs(_f64(Y)[0] - want)
    assert (off <= tol).all(), (float((off - tol).max()), int((off > tol).sum()))
    return Y, rc, flags


def _tokens(rng, T, D, dtype, pad=0):
    import torch

    X = torch.full((T, D + pad), float("nan"), dtype=_t(dtype), device="cuda")
    X[:, :D] = torch.from_numpy(rng.normal(size=(T, D)).astype(np.float32)).cuda()
    return X[:, :D]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,D,F,m", [
    (1, 1, 8, 8, 1), (1, 8, 64, 32, 2), (1, 64, 512, 256, 8), (2, 5, 40, 24, 3),
    (7, 16, 136, 200, 4), (8, 4, 256, 64, 1), (9, 1, 128, 128, 1), (16, 2, 72, 80, 2),
    (17, 3, 1000, 16, 2), (33, 2, 64, 1032, 1), (40, 32, 264, 120, 6), (64, 128, 96, 40, 8),
    (100, 1024, 32, 16, 8), (129, 2, 48, 56, 2), (256, 4, 64, 32, 4), (256, 1, 16, 24, 8),
])
def test_sizes(G, T, E, D, F, m, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    import torch

    X = _tokens(rng, T, D, dtype, 8 if T % 2 else 0)
    W = _weights(rng, E, D, F, dtype)
    if E >= m:
        idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m, renorm=bool(T % 2))
    else:  # more choices than experts: every expert several times
        idx = torch.from_numpy(rng.integers(0, E, (T, m)).astype(np.int32)).cuda()
        resp = torch.rand(T, m, device="cuda")
    _, rc, flags = _check(G, X, idx, resp, *W, act=T % 2)
    assert rc == 0 and flags == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_unused_repeated_and_bad_choices(G, dtype):
    import torch

    rng = np.random.default_rng(3)
    T, E, D, F, m = 21, 6, 88, 104, 4
    X, W = _tokens(rng, T, D, dtype), _weights(rng, E, D, F, dtype)
    idx = rng.integers(0, E, (T, m)).astype(np.int32)
    idx[0] = -1                 # no expert at all
    idx[1] = [2, 2, 2, 2]       # one expert four times
    idx[2] = [-1, 3, -1, 3]
    idx[T - 4:] = -1            # padding behind the last token
    resp = rng.normal(size=(T, m)).astype(np.float32)
    resp[4] = 0.0
    d = [torch.from_numpy(a).cuda() for a in (idx, resp)]
    Y, rc, flags = _check(G, X, *d, *W)
    assert rc == 0 and flags == 0
    assert (Y[0] == 0).all() and (Y[T - 4:] == 0).all()
    idx[5, 1], idx[6, 0] = E, -2
    d[0] = torch.from_numpy(idx).cuda()
    _, rc, flags = _check(G, X, *d, *W)
    assert rc == G.GMM_ERR_INVALID_ARG and flags == G.GMM_DEVFLAG_BAD_INDEX
    idx[:] = -1
    d[0] = torch.from_numpy(idx).cuda()
    Y, _, _ = _check(G, X, *d, *W)
    assert (Y == 0).all()


def test_a_bad_token_stays_alone(G):
    """NaN and infinities in one token, or in unused padding, reach no other token."""
    import torch

    rng = np.random.default_rng(4)
    T, E, D, F, m = 12, 3, 64, 48, 2
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    clean = G.gmm_moe(X, idx, resp, *W)
    X[5, 3], X[7, 0] = float("nan"), float("inf")
    got = G.gmm_moe(X, idx, resp, *W)
    assert torch.isnan(got[5]).all() and not torch.isfinite(got[7]).any()
    keep = [t for t in range(T) if t not in (5, 7)]
    assert torch.equal(got[keep], clean[keep])


def test_strided_output_and_repeated_runs(G):
    import torch

    rng = np.random.default_rng(5)
    T, E, D, F, m = 30, 8, 120, 72, 3
    X, W = _tokens(rng, T, D, "bf16", 16), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    buf = torch.full((T + 2, D + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    Y, _, _ = _check(G, X, idx, resp, *W, out=buf[:T, :D])
    assert (buf[T:] == 3.0).all() and (buf[:, D:] == 3.0).all()
    for _ in range(3):
        assert torch.equal(Y, G.gmm_moe(X, idx, resp, *W))


def test_a_token_does_not_depend_on_its_batch_mates_choices_order(G):
    """The same tokens in another order give the same rows, bit for bit."""
    import torch

    rng = np.random.default_rng(6)
    T, E, D, F, m = 50, 8, 256, 128, 2
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    Y = G.gmm_moe(X, idx, resp, *W)
    perm = torch.randperm(T, device="cuda")
    assert torch.equal(G.gmm_moe(X[perm].contiguous(), idx[perm], resp[perm], *W), Y[perm])


def test_two_streams_and_a_captured_graph(G):
    import torch

    rng = np.random.default_rng(7)
    T, E, D, F, m = 16, 16, 256, 160, 4
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    Z = torch.randn(T, E, device="cuda")
    idx, resp = G.gmm_route(Z, m, renorm=True)
    want = G.gmm_moe(X, idx, resp, *W)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:  # two calls at once, each on a workspace of its own
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(20):
                outs.append(G.gmm_moe(X, idx, resp, *W))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    ws = torch.zeros(G.gmm_moe_workspace_size(G.moe_problem(X, idx, W[1])), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gi, gr = G.gmm_route(Z, m, renorm=True)
        gy = G.gmm_moe(X, gi, gr, *W, ws=ws)
    for _ in range(2):
        Z.normal_()
        X.normal_()
        graph.replay()
        i, r = G.gmm_route(Z, m, renorm=True)
        assert torch.equal(gi, i) and torch.equal(gr, r)
        assert torch.equal(gy, G.gmm_moe(X, i, r, *W))


def test_four_threads_at_once(G):
    """Host threads with a stream and a workspace each."""
    import threading

    import torch

    rng = np.random.default_rng(14)
    T, E, D, F, m = 8, 16, 512, 128, 4
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    want = G.gmm_moe(X, idx, resp, *W)
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = G.gmm_moe(X, idx, resp, *W)
                s.synchronize()
                if not torch.equal(got, want):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_the_first_call_of_a_process_may_be_captured(G):
    """Routing, experts, log probabilities and gradient into a graph before any eager call."""
    import subprocess
    import sys

    code = """
import torch
from soft_clustering_em_b200 import gmm as G
T, E, D, F, m, K = 6, 8, 512, 64, 2, 70_001
X = torch.randn(T, D, device="cuda").bfloat16()
U = torch.randn(E, 2 * F, D, device="cuda").mul_(D ** -0.5).bfloat16()
W = torch.randn(E, D, F, device="cuda").mul_(F ** -0.5).bfloat16()
Z, L = torch.randn(T, E, device="cuda"), torch.randn(3, K, device="cuda")
w = torch.ones(3, device="cuda")
ids = torch.zeros(3, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    i, r = G.gmm_route(Z, m)
    y = G.gmm_moe(X, i, r, U, W)
    q = G.gmm_logprobs(L, ids, m=3)
    d = G.gmm_logprobs_backward(L, ids, q.lse, dlogp=w)
for _ in range(2):
    Z.normal_()
    L.normal_()
    g.replay()
    j, s = G.gmm_route(Z, m)
    p = G.gmm_logprobs(L, ids, m=3)
    assert torch.equal(i, j) and torch.equal(y, G.gmm_moe(X, j, s, U, W))
    assert torch.equal(q.top_idx, p.top_idx) and torch.equal(q.lse, p.lse)
    assert torch.equal(d, G.gmm_logprobs_backward(L, ids, p.lse, dlogp=w))
print("same")
"""
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=240)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]


def test_a_call_on_a_given_stream_owns_its_workspace(G):
    """The workspace made for a call on another stream is not handed out again before it ran."""
    import torch

    rng = np.random.default_rng(14)
    T, E, D, F, m = 7, 9, 256, 128, 2
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    Z = torch.randn(T, E, device="cuda")
    idx, resp = G.gmm_route(Z, m)
    want = G.gmm_moe(X, idx, resp, *W)
    size = G.gmm_moe_workspace_size(G.moe_problem(X, idx, W[1]))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    out = torch.empty_like(X)
    G.gmm_moe(X, idx, resp, *W, out=out, stream=side)
    route = G.gmm_route(Z, m, stream=side)
    others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((o == 255).all()) for o in others)
    assert torch.equal(out, want) and torch.equal(route[0], idx) and torch.equal(route[1], resp)


def test_one_token_of_any_stride(G):
    import torch

    rng = np.random.default_rng(15)
    W = _weights(rng, 3, 64, 32, "bf16")
    big = torch.zeros(2, 1001, dtype=torch.bfloat16, device="cuda")
    big[:, :64] = _tokens(rng, 2, 64, "bf16")
    idx, resp = G.gmm_route(torch.randn(1, 3, device="cuda"), 2)
    X, out = big[:1, :64], torch.empty(2, 77, dtype=torch.bfloat16, device="cuda")[:1, :64]
    assert torch.equal(G.gmm_moe(X, idx, resp, *W, out=out),
                       G.gmm_moe(X.contiguous(), idx, resp, *W))


def test_a_short_budget_times_out_and_the_next_call_is_exact(G):
    import torch

    rng = np.random.default_rng(12)
    T, E, D, F, m = 20, 12, 512, 256, 3
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    ws = torch.zeros(G.gmm_moe_workspace_size(G.moe_problem(X, idx, W[1])), dtype=torch.uint8,
                     device="cuda")
    try:
        G.gmm_set_wait_budget(1)  # 1 ns: a wait that is not over at the second look gives up
        G.gmm_moe(X, idx, resp, *W, ws=ws)
        rc, flags = G.gmm_device_status(ws)
    finally:
        G.gmm_set_wait_budget(0)
    assert rc == G.GMM_ERR_TIMEOUT and flags == G.GMM_DEVFLAG_WAIT_TIMEOUT
    _, rc, flags = _check(G, X, idx, resp, *W)
    assert rc == 0 and flags == 0


@pytest.mark.parametrize("D,F", [(64, 64), (256, 128), (512, 512)])
def test_a_short_budget_with_every_copy_on_its_way(G, D, F):
    """Streams no longer than the ring: no copy waits for a stage, the products give up.  The CTAs
    end after their copies have landed, so the calls right behind them are exact."""
    import torch

    rng = np.random.default_rng(D)
    X, W = _tokens(rng, 5, D, "f16"), _weights(rng, 3, D, F, "f16")
    idx, resp = G.gmm_route(torch.randn(5, 3, device="cuda"), 2)
    want = G.gmm_moe(X, idx, resp, *W)
    p = G.moe_problem(X, idx, W[1])
    for _ in range(20):
        ws = torch.zeros(G.gmm_moe_workspace_size(p), dtype=torch.uint8, device="cuda")
        ws2 = torch.zeros_like(ws)
        try:
            G.gmm_set_wait_budget(1)
            G.gmm_moe(X, idx, resp, *W, ws=ws)
        finally:
            G.gmm_set_wait_budget(0)
        got = G.gmm_moe(X, idx, resp, *W, ws=ws2)
        assert G.gmm_device_status(ws2) == (0, 0)
        assert torch.equal(got, want)


@pytest.mark.parametrize("T,E,D,F,m", [(256, 2, 1024, 512, 2), (70, 3, 264, 712, 2),
                                       (200, 16, 2048, 64, 4), (31, 160, 136, 72, 8)])
def test_longer_streams(G, T, E, D, F, m):
    """Many jobs per CTA, rings that wrap, experts of several column groups, unequal tails."""
    import torch

    rng = np.random.default_rng(T)
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    Y, rc, flags = _check(G, X, idx, resp, *W)
    assert rc == 0 and flags == 0
    for _ in range(5):
        assert torch.equal(Y, G.gmm_moe(X, idx, resp, *W))


def test_weights_of_other_experts_do_not_reach_a_token(G):
    """NaN and infinities in the weights of an expert reach the tokens that chose it alone."""
    import torch

    rng = np.random.default_rng(13)
    T, E, D, F, m = 18, 5, 128, 96, 2
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    idx, resp = G.gmm_route(torch.randn(T, E, device="cuda"), m)
    clean = G.gmm_moe(X, idx, resp, *W)
    W[0][3, 5, 7] = float("nan")
    W[1][3, 64:, :] = float("inf")
    got = G.gmm_moe(X, idx, resp, *W)
    chose = (idx == 3).any(1)
    assert chose.any() and not chose.all()
    assert torch.equal(got[~chose], clean[~chose])
    assert torch.isnan(got[chose]).any(1).all()


def test_weights_of_more_than_32_bits(G):
    """Experts 2^31 elements and 2^32 bytes into the weights, against the same ones by themselves
    (one choice per token: no sum whose order could differ)."""
    import torch

    rng = np.random.default_rng(16)
    E, D, F = 300, 2048, 2048
    some = [0, 131, 262, 299]
    X, (U, V) = _tokens(rng, 6, D, "bf16"), _weights(rng, len(some), D, F, "bf16")
    big_u = torch.zeros(E, 2 * F, D, dtype=U.dtype, device="cuda")
    big_v = torch.zeros(E, D, F, dtype=U.dtype, device="cuda")
    big_u[some], big_v[some] = U, V
    few = torch.tensor([[0], [1], [2], [3], [3], [2]], dtype=torch.int32, device="cuda")
    many = torch.tensor(some, dtype=torch.int32, device="cuda")[few.long()]
    resp = torch.rand(6, 1, device="cuda")
    got = G.gmm_moe(X, many, resp, big_u, big_v)
    assert torch.equal(got, G.gmm_moe(X, few, resp, U, V)) and bool((got != 0).any(1).all())


def test_no_tokens(G):
    import torch

    W = _weights(np.random.default_rng(8), 2, 16, 8, "bf16")
    X = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    Y = G.gmm_moe(X, idx, torch.empty(0, 2, device="cuda"), *W)
    assert Y.shape == (0, 16)


def test_experts_of_a_mixture(G):
    """Points go to the experts of their mixture components: gmm_assign_topm's assignment is
    gmm_moe's."""
    wl = synth.WORKLOADS["bf16stream"]
    import torch

    N, K, m = 200, 64, 2
    data, _ = synth.make_data(wl, 4096)
    Xd = torch.from_numpy(data.view(np.int16)).view(torch.bfloat16).cuda()
    w, mu, var = G.gmm_init(Xd, 3, K)
    G.gmm_fit(Xd, w, mu, var, iters=3)
    idx, resp = G.gmm_assign_topm(Xd[:N].contiguous(), w, mu, var, m)
    W = _weights(np.random.default_rng(9), K, wl.D, 48, "bf16")
    _, rc, flags = _check(G, Xd[:N].contiguous(), idx, resp, *W)
    assert rc == 0 and flags == 0


def test_route_experts_head_and_gradient_together(G):
    """A layer and a head as they are used: route, experts, vocabulary logits, the labels' log
    probabilities, and the logits' gradient in place."""
    import torch

    rng = np.random.default_rng(10)
    T, E, D, F, m, V = 24, 16, 128, 96, 4, 5003
    X, W = _tokens(rng, T, D, "bf16"), _weights(rng, E, D, F, "bf16")
    gate = torch.from_numpy(rng.normal(size=(E, D)).astype(np.float32)).cuda() / np.sqrt(D)
    head = torch.from_numpy(rng.normal(size=(V, D)).astype(np.float32)).cuda().bfloat16()
    ids = rng.integers(0, V, T).astype(np.int32)
    ids[::6] = -1
    ids_d = torch.from_numpy(ids).cuda()
    idx, resp = G.gmm_route(X.float() @ gate.T, m, renorm=True)
    Y, rc, flags = _check(G, X, idx, resp, *W)
    assert rc == 0 and flags == 0
    logits = (X + Y) @ head.T
    z = logits.float().cpu().numpy()
    r = G.gmm_logprobs(logits, ids_d, m=5)
    logp, H, lse, ti, tl = P.logprobs(z, ids, 5)
    np.testing.assert_array_equal(r.top_idx.cpu().numpy(), ti)
    # log probabilities to u (2 max|z| + 3 * 104 + 75 + 20) + roundings, as in the rows' own tests
    tol = 2.0 ** -24 * (6 * np.abs(z).max() + 3 * 104 + 75 + 20 + 4 * np.abs(tl).max())
    for got, want in ((r.logp, logp), (r.lse, lse), (r.top_logp, tl)):
        np.testing.assert_allclose(_f64(got)[0], want, rtol=0, atol=tol)
    w = -torch.ones(T, device="cuda") / T
    want = P.gradient(z, ids, _f64(r.lse)[0], None, _f64(w)[0], None, None, None, None)
    g = G.gmm_logprobs_backward(logits, ids_d, r.lse, dlogp=w, out=logits)
    # half a step of bf16, and p to tol in relation
    np.testing.assert_array_less(np.abs(_f64(g)[0] - want),
                                 np.abs(want) * (2.0 ** -8 + 2 * tol) + 2.0 ** -24 / T)
