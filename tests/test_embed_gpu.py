"""gmm_embed and gmm_embed_backward on the GPU against oracle/assignments.py.

Tolerances, for u = 2^-24 and sums of c float32 terms one after another: (c + 4) u times the sum of
the terms' magnitudes (each product and each addition rounds once, and the scale), then half a step
of the result's type relative to the value, and half its smallest step (float16 2^-25, bfloat16
2^-134).  A class that is named n times is summed in chunks of 16 to 128, the chunks' sums by 8 to
256 groups in turn, and those by halves: c <= min(n, 128) + n / 128 + 8.  dresp: a lane adds up at
most D / 8 terms, then up to 12 levels.
"""
import numpy as np
import pytest

from oracle import assignments as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


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


def _rows(rng, N, D, dtype, pad=0, shift=0):
    """N x D numbers in rows of D + pad, `shift` entries into a buffer of NaN; and their values."""
    import torch

    buf = torch.full((N * (D + pad) + shift + 64,), float("nan"), dtype=_t(dtype), device="cuda")
    x = buf[shift:shift + N * (D + pad)].view(N, D + pad)[:, :D]
    x.copy_(torch.from_numpy(rng.normal(size=(N, D)).astype(np.float32)))
    return x, x.double().cpu().numpy()


def _assignment(rng, N, m, K, weights):
    import torch

    idx = rng.integers(0, K, (N, m)).astype(np.int32)
    idx[rng.random((N, m)) < 0.1] = -1
    if N > 4:
        idx[1] = -1               # a row without choices
        idx[2] = idx[0]           # the same choices in two rows
        idx[3] = idx[3, 0]        # and the same choice m times in one
        idx[-1] = K - 1
    r = rng.normal(size=(N, m)).astype(np.float32) if weights else None
    return (torch.from_numpy(idx).cuda(), None if r is None else torch.from_numpy(r).cuda(),
            idx, r)


def _near(got, want, tol, what=""):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), (what, off.max(), np.unravel_index(off.argmax(), off.shape))


def _depth(named):
    return (np.minimum(named, 128) + named / 128 + 8)[:, None]


SHAPES = [  # N, m, K, D, pad, shift
    (1, 1, 1, 1, 0, 0), (1, 1, 50, 8, 0, 0), (3, 2, 7, 5, 0, 0), (33, 1, 100, 64, 0, 0),
    (257, 3, 300, 96, 8, 0), (500, 8, 40, 24, 0, 1), (1000, 1, 2000, 257, 3, 0),
    (70, 2, 10, 2048, 0, 0), (64, 1, 9, 8200, 0, 0), (900, 4, 5000, 100, 4, 2),
    (5000, 1, 3, 16, 0, 0), (2, 1, 70000, 40, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,m,K,D,pad,shift", SHAPES)
def test_lookup(G, N, m, K, D, pad, shift, dtype):
    rng = np.random.default_rng(N + D)
    W, w = _rows(rng, K, D, dtype, pad, shift)
    idx, resp, i, r = _assignment(rng, N, m, K, m > 1 or N % 2)
    want, size = A.embed(w, i, r, 1.25)
    tol = (m + 4) * U * size + HALF[dtype] * np.abs(want) + LEAST[dtype]
    _near(G.gmm_embed(W, idx, resp, scale=1.25), want, tol)
    if m == 1:
        one = [None if t is None else t[:, 0].contiguous() for t in (idx, resp)]
        _near(G.gmm_embed(W, *one, scale=1.25), want, tol)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("N,m,K,D,pad,shift", SHAPES)
def test_gradient(G, N, m, K, D, pad, shift, dtype, out, add):
    rng = np.random.default_rng(N + D + 1)
    dY, dy = _rows(rng, N, D, dtype, pad, shift)
    idx, resp, i, r = _assignment(rng, N, m, K, m > 1 or N % 2)
    dW, old = _rows(rng, K, D, out, pad, shift)
    want, size, named = A.embed_backward(dy, i, K, r, 0.75)
    tol = (_depth(named) + 4) * U * size
    if add:
        want = want + old
        tol = tol + U * np.abs(want)
    tol = tol + HALF[out] * np.abs(want) + LEAST[out]
    before = dW.clone()
    got, none = G.gmm_embed_backward(dY, idx, K, resp, scale=0.75, out=dW, accumulate=add)
    assert none is None and got is dW
    if add:  # rows that nothing names are not touched
        tol[named == 0] = 0
    _near(dW, want, tol)
    again = before.clone()
    again, _ = G.gmm_embed_backward(dY, idx, K, resp, scale=0.75, out=again, accumulate=add)
    if not (pad or shift):
        assert (again == dW).all()  # from run to run


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,m,K,D,pad,shift", SHAPES)
def test_gradient_of_the_weights(G, N, m, K, D, pad, shift, dtype):
    rng = np.random.default_rng(N + D + 2)
    dY, dy = _rows(rng, N, D, dtype, pad, shift)
    W, w = _rows(rng, K, D, dtype, pad, shift)
    idx, resp, i, r = _assignment(rng, N, m, K, True)
    dW, dresp = G.gmm_embed_backward(dY, idx, K, resp, W=W, scale=0.75)
    want, size = A.embed_dresp(dy, w, i, 0.75)
    _near(dresp, want, (D / 8 + 12) * U * size)
    want, size, named = A.embed_backward(dy, i, K, r, 0.75)
    _near(dW, want, (_depth(named) + 4) * U * size + HALF[dtype] * np.abs(want) + LEAST[dtype])


@pytest.mark.parametrize("N,K,D,how", [
    (20000, 5, 64, "one"), (20000, 100, 40, "two"), (300_000, 1000, 8, "skewed"),
    (70_000, 1 << 21, 4, "skewed"), (1000, 1 << 20, 3, "skewed"), (131_073, 30, 16, "one"),
    (2048, 1023, 8, "all"), (4096, 1024, 8, "all"),
])
def test_lists_of_all_lengths(G, N, K, D, how):
    """A class that has every choice, runs that end on a chunk's border, one to three digits."""
    import torch

    rng = np.random.default_rng(N)
    dY, dy = _rows(rng, N, D, "f32")
    i = {"one": np.full(N, K - 1), "two": np.where(np.arange(N) < N // 2, 3, 97),
         "skewed": np.minimum((K ** rng.random(N)).astype(np.int64) - 1, K - 1),
         "all": np.arange(N)[::-1] % K}[how].astype(np.int32)
    got, _ = G.gmm_embed_backward(dY, torch.from_numpy(i).cuda(), K)
    want, size, named = A.embed_backward(dy, i, K)
    _near(got, want, (_depth(named) + 4) * U * size + HALF["f32"] * np.abs(want))
    got2, _ = G.gmm_embed_backward(dY, torch.from_numpy(i).cuda(), K)
    assert torch.equal(got, got2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,pad,shift", [(40, 8, 0), (41, 7, 0), (40, 3, 1), (300, 1, 0)])
def test_results_in_rows_of_another_tensor(G, D, pad, shift, dtype):
    """Aligned tables into rows that start anywhere and the other way; what lies between stays."""
    import torch

    rng = np.random.default_rng(D + pad)
    N, K = 70, 30
    for table in ((pad, shift), (0, 0)):
        W, w = _rows(rng, K, D, dtype, *table)
        idx, resp, i, r = _assignment(rng, N, 2, K, True)
        buf = torch.full((N * (D + pad) + shift + 64,), 7.0, dtype=_t(dtype), device="cuda")
        out = buf[shift:shift + N * (D + pad)].view(N, D + pad)[:, :D]
        assert G.gmm_embed(W, idx, resp, out=out) is out
        want, size = A.embed(w, i, r)
        _near(out, want, 6 * U * size + HALF[dtype] * np.abs(want) + LEAST[dtype])
        out.fill_(7.0)
        assert (buf == 7).all()


def test_nothing_to_look_up(G):
    import torch

    W = torch.ones(5, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert G.gmm_embed(W, none).shape == (0, 8)
    out = torch.full((5, 8), 3.0, device="cuda")
    G.gmm_embed_backward(W[:0], none, 5, out=out, accumulate=True)
    assert (out == 3).all()
    G.gmm_embed_backward(W[:0], none, 5, out=out)
    assert (out == 0).all()
    idx = torch.full((7,), -1, dtype=torch.int32, device="cuda")
    assert (G.gmm_embed(W, idx) == 0).all()
    G.gmm_embed_backward(torch.full((7, 8), float("nan"), device="cuda"), idx, 5, out=out)
    assert (out == 0).all()


def test_bad_indices_are_left_out_and_told(G):
    import torch

    W = torch.randn(6, 16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = torch.tensor([[0, 5], [2, -1]], dtype=torch.int32, device="cuda")
    G.gmm_embed(W, good, dev_flags=flags)
    G.gmm_embed_backward(W[:2], good, 6, W=W, dev_flags=flags)
    assert flags.item() == 0
    bad = torch.tensor([[0, 6], [-2, 2]], dtype=torch.int32, device="cuda")
    Y = G.gmm_embed(W, bad, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    assert torch.equal(Y, W[[0, 2]])
    flags.zero_()
    dW, dresp = G.gmm_embed_backward(W[:2], bad, 6, W=W, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    assert torch.equal(dW[[0, 2]], W[[0, 1]]) and (dW[[1, 3, 4, 5]] == 0).all()
    assert (dresp[[0, 1], [1, 0]] == 0).all()


def test_a_nan_reaches_only_what_it_is_part_of(G):
    import torch

    W = torch.ones(4, 24, device="cuda", dtype=torch.bfloat16)
    W[1] = float("nan")
    W[3] = float("inf")
    idx = torch.tensor([[0, 2], [1, 2], [-1, 0], [3, 0]], dtype=torch.int32, device="cuda")
    Y = G.gmm_embed(W, idx)
    assert (Y[0] == 2).all() and Y[1].isnan().all() and (Y[2] == 1).all() and Y[3].isinf().all()
    dY = torch.ones(4, 24, device="cuda")
    dY[1] = float("nan")
    dW, _ = G.gmm_embed_backward(dY, idx, 4)
    assert (dW[0] == 3).all() and dW[1].isnan().all() and dW[2].isnan().all() and (dW[3] == 1).all()


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("K", [1, 2, 1023, 1024, 1 << 20])
@pytest.mark.parametrize("M", [31, 127, 128, 129, 1023, 1024, 1025, 16_385, (1 << 17) - 1, 1 << 17,
                               (1 << 17) + 1])
def test_where_the_ways_to_sum_change(G, M, K, add):
    """Numbers of choices beside those at which another path is taken, and digits of the sort; half
    of the choices name one class.  Whole numbers: the sums are exact."""
    import torch

    D = 9
    g = torch.Generator(device="cuda").manual_seed(M + K)
    idx = torch.randint(-1, K, (M,), generator=g, device="cuda", dtype=torch.int32)
    idx[::2] = K - 1
    dY = torch.randint(-8, 9, (M, D), generator=g, device="cuda").float()
    out = torch.full((K, D), 3.0, device="cuda")
    G.gmm_embed_backward(dY, idx, K, out=out, accumulate=add)
    want = torch.full((K + 1, D), 3.0 if add else 0.0, device="cuda", dtype=torch.float64)
    want.index_add_(0, torch.where(idx < 0, K, idx).long(), dY.double())
    assert torch.equal(out.double(), want[:K])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 128, 129, 591, 592, 593, 2000])
@pytest.mark.parametrize("D", [8, 256, 264, 512, 520, 1031])
def test_where_the_ways_to_multiply_change(G, N, D, dtype):
    """Rows and widths beside those at which the weights' gradient takes other lanes."""
    rng = np.random.default_rng(N + D)
    for m in (1, 2, 3, 5):
        dY, dy = _rows(rng, N, D, dtype)
        W, w = _rows(rng, 50, D, dtype)
        idx, resp, i, _ = _assignment(rng, N, m, 50, True)
        _, dresp = G.gmm_embed_backward(dY, idx, 50, resp, W=W)
        want, size = A.embed_dresp(dy, w, i)
        _near(dresp, want, (D / 8 + 12) * U * size)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,D,pad,shift", [(60_000, 1000, 0, 0), (60_000, 1000, 8, 0),
                                           (150_001, 301, 0, 0), (150_001, 301, 2, 1),
                                           (1_000_003, 64, 0, 0)])
@pytest.mark.parametrize("M", [1, 3000, 150_000])
def test_large_tables_are_written_throughout(G, K, D, pad, shift, dtype, M):
    """Ones summed are counts (whole numbers up to 256 in bfloat16), everywhere else zeros: also in
    the rows that are written after the sort, and not between the rows."""
    import torch

    idx = torch.randint(0, K, (M,), device="cuda", dtype=torch.int32)
    idx[::7] = K - 1 - idx[::7] // 1000
    buf = torch.full((K * (D + pad) + shift + 64,), float("nan"), dtype=_t(dtype), device="cuda")
    out = buf[shift:shift + K * (D + pad)].view(K, D + pad)[:, :D]
    dY = torch.ones(1, D, dtype=_t(dtype), device="cuda").expand(M, D).contiguous()
    G.gmm_embed_backward(dY, idx, K, out=out)
    want = torch.bincount(idx.long(), minlength=K).to(_t(dtype))
    assert torch.equal(out, want[:, None].expand(K, D))
    assert buf.isnan().sum() == buf.numel() - K * D


def test_tables_beyond_32_bits(G):
    """Rows whose offsets pass 2^32 bytes and 2^31 elements."""
    import torch

    K, D = 70_000, 32_768  # 2.3e9 bfloat16
    W = torch.zeros(K, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.tensor([K - 1, 0, 65_537], dtype=torch.int32, device="cuda")
    W[idx.long()] = torch.randn(3, D, device="cuda").bfloat16()
    Y = G.gmm_embed(W, idx)
    assert torch.equal(Y, W[idx.long()])
    dW, _ = G.gmm_embed_backward(Y, idx, K, out=W.fill_(1.0))
    assert torch.equal(dW[idx.long()], Y)
    assert dW.count_nonzero() == Y.count_nonzero()


def test_a_class_that_millions_of_choices_name(G):
    """Alike terms, whose roundings in a running sum all go one way: 128 of a chunk, 8 chunks' sums,
    8 of those, then 64 bits, 3 halves (32 lanes a row) and the result."""
    import torch

    N, D = 1 << 23, 136
    dY = torch.ones(N, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(N, dtype=torch.int32, device="cuda")
    resp = torch.full((N,), 0.7, device="cuda")
    dW = torch.empty(2, D, device="cuda")
    G.gmm_embed_backward(dY, idx, 2, resp, out=dW)
    want = N * float(np.float32(0.7))
    assert (dW[1] == 0).all()
    assert (dW[0].double() / want - 1).abs().max() <= (128 + 8 + 8 + 4) * U


def test_an_infinite_term_among_millions(G):
    """The sum of a class with infinities is infinite, in a long run too, or NaN for both signs."""
    import torch

    N, D = 300_000, 8
    dY = torch.ones(N, D, device="cuda")
    dY[100, 0], dY[200_000, 1], dY[5, 2], dY[299_999, 2] = np.inf, -np.inf, np.inf, -np.inf
    idx = torch.zeros(N, dtype=torch.int32, device="cuda")
    dW, _ = G.gmm_embed_backward(dY, idx, 1)
    assert dW[0, 0] == np.inf and dW[0, 1] == -np.inf and dW[0, 2].isnan()
    assert (dW[0, 3:] == N).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,m,D,pad", [(0, 1, 8, 0), (1, 1, 40, 0), (64, 2, 96, 0), (64, 3, 41, 3),
                                       (129, 1, 2048, 0), (700, 2, 520, 0), (5000, 4, 64, 8),
                                       (140_000, 1, 16, 0)])
def test_the_gradient_of_the_weights_alone(G, N, m, D, pad, dtype):
    """What the call for both gives, bit for bit; no table's gradient and no workspace."""
    import torch

    K = 300
    rng = np.random.default_rng(N + D)
    W, _ = _rows(rng, K, D, dtype, pad)
    dY, _ = _rows(rng, N, D, dtype, pad)
    idx, resp, _, _ = _assignment(rng, N, m, K, True)
    _, want = G.gmm_embed_backward(dY, idx, K, resp, W=W, scale=0.7)
    none, got = G.gmm_embed_backward(dY, idx, K, resp, W=W, scale=0.7, table=False)
    assert none is None and got.shape == idx.shape and torch.equal(got, want)
    again = torch.full_like(want, float("nan"))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = G.embed_problem(idx, K, 0.7, W.stride(0), dY)
    assert G.load_library().gmm_embed_backward(
        p, dY.data_ptr(), idx.data_ptr(), resp.data_ptr(), W.data_ptr(), None, 0, 0, 0,
        again.data_ptr(), flags.data_ptr(), None, 0,
        torch.cuda.current_stream().cuda_stream) == G.GMM_OK
    assert torch.equal(again, want) and flags.item() == 0


def test_the_gradient_of_the_weights_alone_captured_and_refused(G):
    import torch

    dY, W = torch.randn(50, 24, device="cuda"), torch.randn(9, 24, device="cuda")
    idx = torch.randint(0, 9, (50, 2), dtype=torch.int32, device="cuda")
    resp = torch.rand(50, 2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, got = G.gmm_embed_backward(dY, idx, 9, resp, W=W, table=False)
    dY.normal_()
    idx[7, 1] = 40
    graph.replay()
    torch.cuda.synchronize()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = G.gmm_embed_backward(dY, idx, 9, resp, W=W, dev_flags=flags, table=False)[1]
    assert torch.equal(got, want) and got[7, 1] == 0 and flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    for kw in (dict(W=None), dict(W=W, out=torch.zeros_like(W)), dict(W=W, accumulate=True)):
        with pytest.raises(ValueError):
            G.gmm_embed_backward(dY, idx, 9, resp, table=False, **kw)


def test_captured_and_on_another_stream(G):
    import torch

    rng = np.random.default_rng(3)
    N, K, D = 300, 500, 64
    dY, _ = _rows(rng, N, D, "f32")
    W, _ = _rows(rng, K, D, "f32")
    idx = torch.from_numpy(rng.integers(0, K, N).astype(np.int32)).cuda()
    want = G.gmm_embed(W, idx), G.gmm_embed_backward(dY, idx, K)[0]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    got = G.gmm_embed(W, idx, stream=other), G.gmm_embed_backward(dY, idx, K, stream=other)[0]
    other.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    p = G.embed_problem(idx, K, 1.0, D, dY)
    ws = torch.empty(G.gmm_embed_workspace_size(p), dtype=torch.uint8, device="cuda")
    graph, Y, dW = torch.cuda.CUDAGraph(), torch.empty_like(want[0]), torch.empty_like(want[1])
    with torch.cuda.graph(graph):
        G.gmm_embed(W, idx, out=Y)
        G.gmm_embed_backward(dY, idx, K, out=dW, ws=ws)
    for seed in (4, 5):
        new = torch.from_numpy(np.random.default_rng(seed).integers(0, K, N).astype(np.int32))
        idx.copy_(new)
        ws.fill_(255)  # any content
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, W[idx.long()])
        assert torch.equal(dW, G.gmm_embed_backward(dY, idx, K)[0])


@pytest.mark.parametrize("bad", ["0.5", b"0.5", None])
def test_a_scale_that_is_no_number_is_refused(G, bad):
    import torch

    W, idx = torch.ones(4, 8, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: G.gmm_embed(W, idx, scale=bad),
                 lambda: G.gmm_embed_backward(W[:2], idx, 4, scale=bad),
                 lambda: G.gmm_route_loss(W[:2], idx[:, None], scale=bad),
                 lambda: G.gmm_logprobs(W, scale=bad), lambda: G.gmm_route(W, 2, scale=bad)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("N,m", [(500, 2), (20_000, 1), (70_000, 2)])
def test_inputs_written_by_the_kernel_before(G, N, m):
    """What goes on beside the sort sees what came just before it, replayed too, with a workspace of
    any content; each replay has inputs of its own."""
    import torch

    K, D = 900, 64
    g = torch.Generator(device="cuda").manual_seed(N)
    dYs = torch.randn(6, N, D, device="cuda", generator=g)
    ids = torch.randint(-1, K, (6, N, m), device="cuda", generator=g, dtype=torch.int32)
    resp = torch.rand(N, m, device="cuda", generator=g)
    Ws = torch.randn(6, K, D, device="cuda", generator=g)
    dY, idx, W, dW = dYs[0].clone(), ids[0].clone(), Ws[0].clone(), torch.empty(K, D, device="cuda")
    ws = torch.empty(G.gmm_embed_workspace_size(G.embed_problem(idx, K, 1.0, D, dY)),
                     dtype=torch.uint8, device="cuda")
    want = []
    for i in range(6):
        torch.cuda.synchronize()
        want.append(G.gmm_embed_backward(dYs[i], ids[i], K, resp, W=Ws[i]))
    from_dY, from_idx, from_W = dYs[0].clone(), ids[0].clone(), Ws[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.copy_(from_W)
        idx.copy_(from_idx)
        dY.copy_(from_dY)
        _, got = G.gmm_embed_backward(dY, idx, K, resp, W=W, out=dW, ws=ws)
    for i in (1, 2, 3, 4, 5, 1, 0):
        if i == 3:
            ws.fill_(255)
        for t, v in ((from_dY, dYs[i]), (from_idx, ids[i]), (from_W, Ws[i])):
            t.copy_(v)
        graph.replay()
        have = dW.clone(), got.clone()
        graph.replay()
        assert all(torch.equal(a, b) and torch.equal(c, b)
                   for a, b, c in zip(have, want[i], (dW, got)))


def test_refusals(G):
    import torch

    W = torch.zeros(6, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    dY = torch.zeros(4, 8, device="cuda")
    for bad in (lambda: G.gmm_embed(W, idx.long()), lambda: G.gmm_embed(W, idx.cpu()),
                lambda: G.gmm_embed(W.double(), idx), lambda: G.gmm_embed(W.t(), idx),
                lambda: G.gmm_embed(W, idx, torch.zeros(4, device="cuda")),
                lambda: G.gmm_embed(W, idx.t()), lambda: G.gmm_embed(W, idx, out=dY.half()),
                lambda: G.gmm_embed(W, idx[0, 0]),
                lambda: G.gmm_embed_backward(dY, idx[:3], 6),
                lambda: G.gmm_embed_backward(dY, idx, 6, W=W.half()),
                lambda: G.gmm_embed_backward(dY, idx, 7, W=W),
                lambda: G.gmm_embed_backward(dY, idx, 6, accumulate=True),
                lambda: G.gmm_embed_backward(dY, idx, 6, out=W.half()),
                lambda: G.gmm_embed_backward(dY, idx, 6, out=W[:5]),
                lambda: G.gmm_embed_backward(dY[:, :1].expand(4, 8), idx, 6)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(G.GmmError):
        G.gmm_embed(W, torch.zeros(4, 9, dtype=torch.int32, device="cuda"))
    with pytest.raises(G.GmmError):
        G.gmm_embed(W, idx, scale=float("nan"))
    with pytest.raises(G.GmmError):  # one row for all
        G.gmm_embed_backward(dY[:1].expand(4, 8), idx, 6)
    with pytest.raises(G.GmmError):
        G.gmm_embed_backward(dY, idx, 6, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
