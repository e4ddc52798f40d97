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
