"""What a caller of gmm_moe sees of a call that went wrong."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from soft_clustering_em_b200 import build
    from soft_clustering_em_b200 import gmm

    build.build()
    gmm.load_library()
    return gmm


def _layer(G, T, E, D, F, m, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, D, generator=g, device="cuda").to(dtype)
    W_up = (torch.randn(E, 2 * F, D, generator=g, device="cuda") * D ** -0.5).to(dtype)
    W_down = (torch.randn(E, D, F, generator=g, device="cuda") * F ** -0.5).to(dtype)
    idx, resp = G.gmm_route(torch.randn(T, E, generator=g, device="cuda"), m)
    return X, idx, resp, W_up, W_down


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,D,F,m", [(20, 12, 512, 256, 3), (1, 8, 2048, 512, 4),
                                       (200, 4, 1024, 712, 2)])
def test_results_that_a_wait_gave_up_on_are_nan(G, T, E, D, F, m, dtype):
    """An entry of a call that timed out is exact or NaN, never something else."""
    args = _layer(G, T, E, D, F, m, dtype)
    want = G.gmm_moe(*args)
    torch.cuda.synchronize()
    lost = 0
    for budget in (1, 1, 2000, 5000, 20_000):  # ns: from nearly all to hardly any
        ws = torch.zeros(G.gmm_moe_workspace_size(G.moe_problem(args[0], args[1], args[4])),
                         dtype=torch.uint8, device="cuda")
        try:
            G.gmm_set_wait_budget(budget)
            Y = G.gmm_moe(*args, ws=ws)
            rc, flags = G.gmm_device_status(ws)
        finally:
            G.gmm_set_wait_budget(0)
        nan = torch.isnan(Y)
        assert ((Y == want) | nan).all()
        assert bool(nan.any()) == (flags != 0)
        assert (rc, flags) in ((0, 0), (G.GMM_ERR_TIMEOUT, G.GMM_DEVFLAG_WAIT_TIMEOUT))
        lost += int(nan.any())
    assert lost >= 2
    assert torch.equal(G.gmm_moe(*args), want)


def test_dev_flags_without_a_workspace(G):
    X, idx, resp, W_up, W_down = _layer(G, 9, 6, 128, 64, 2)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = G.gmm_moe(X, idx, resp, W_up, W_down, dev_flags=flags)
    assert flags.item() == 0
    idx = idx.clone()
    idx[3, 1] = 6
    got = G.gmm_moe(X, idx, resp, W_up, W_down, dev_flags=flags)
    assert flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    keep = [t for t in range(9) if t != 3]
    assert torch.equal(got[keep], want[keep])
    try:
        G.gmm_set_wait_budget(1)
        G.gmm_moe(X, idx, resp, W_up, W_down, dev_flags=flags)
        torch.cuda.synchronize()
    finally:
        G.gmm_set_wait_budget(0)
    both = G.GMM_DEVFLAG_BAD_INDEX | G.GMM_DEVFLAG_WAIT_TIMEOUT
    assert flags.item() == both  # bits are OR-ed in, never cleared
    idx[3, 1] = -1
    G.gmm_moe(X, idx, resp, W_up, W_down, dev_flags=flags)
    assert flags.item() == both


def test_dev_flags_with_a_workspace_on_a_stream_and_in_a_graph(G):
    X, idx, resp, W_up, W_down = _layer(G, 9, 6, 128, 64, 2, seed=1)
    ws = torch.zeros(G.gmm_moe_workspace_size(G.moe_problem(X, idx, W_down)), dtype=torch.uint8,
                     device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = idx.clone()
    bad[0, 0] = -5
    want = G.gmm_moe(X, bad, resp, W_up, W_down)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = G.gmm_moe(X, bad, resp, W_up, W_down, ws=ws, stream=side, dev_flags=flags)
    side.synchronize()
    assert torch.equal(got, want) and flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    assert G.gmm_device_status(ws) == (G.GMM_ERR_INVALID_ARG, G.GMM_DEVFLAG_BAD_INDEX)
    flags.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = G.gmm_moe(X, bad, resp, W_up, W_down, dev_flags=flags)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and flags.item() == G.GMM_DEVFLAG_BAD_INDEX
    flags.zero_()
    bad.copy_(idx)
    graph.replay()
    torch.cuda.synchronize()
    assert flags.item() == 0 and torch.equal(y, G.gmm_moe(X, idx, resp, W_up, W_down))


def test_dev_flags_are_checked(G):
    X, idx, resp, W_up, W_down = _layer(G, 3, 2, 16, 8, 1)
    with pytest.raises(TypeError):
        G.gmm_moe(X, idx, resp, W_up, W_down,
                  dev_flags=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        G.gmm_moe(X, idx, resp, W_up, W_down,
                  dev_flags=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        G.gmm_moe(X, idx, resp, W_up, W_down, dev_flags=torch.zeros(1, dtype=torch.int32))
