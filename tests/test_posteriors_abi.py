"""gmm_logprobs, gmm_logprobs_backward, gmm_route and gmm_moe refuse bad arguments on the host,
before anything is enqueued (no GPU needed), and the binding refuses tensors it cannot pass on."""
import ctypes

import pytest
import torch

from soft_clustering_em_b200 import gmm as G

P = ctypes.c_void_p
BAD, UNSUP, WS = G.GMM_ERR_INVALID_ARG, G.GMM_ERR_UNSUPPORTED, G.GMM_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from soft_clustering_em_b200 import build

    build.build()
    return G.load_library()


def rows(N=10, ld=8, K=8, dtype=G.GMM_F32, scale=1.0):
    return ctypes.byref(G.gmm_rows(N, ld, K, dtype, scale))


BAD_ROWS = [
    (dict(N=-1), BAD), (dict(K=0), BAD), (dict(ld=7), BAD), (dict(dtype=3), BAD),
    (dict(dtype=-1), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(K=(1 << 24) + 1, ld=1 << 25), UNSUP), (dict(N=(1 << 40) + 1), UNSUP),
    (dict(N=1 << 40, ld=1 << 30), UNSUP),
]


def logprobs(lib, r=None, Z=16, ids=16, m=2, logp=16, H=16, lse=16, ti=16, tv=16):
    return lib.gmm_logprobs(r or rows(), P(Z), P(ids), m, P(logp), P(H), P(lse), P(ti), P(tv),
                            P(0), P(0))


def backward(lib, r=None, Z=16, ids=16, lse=16, H=16, dlogp=16, dH=16, dlse=16, m=2, ti=16,
             dtop=16, dZ=32, ldd=8):
    return lib.gmm_logprobs_backward(r or rows(), P(Z), P(ids), P(lse), P(H), P(dlogp), P(dH),
                                     P(dlse), m, P(ti), P(dtop), P(dZ), ldd, P(0), P(0))


def route(lib, r=None, Z=16, m=2, renorm=1, idx=16, resp=16):
    return lib.gmm_route(r or rows(), P(Z), m, renorm, P(idx), P(resp), P(0), P(0))


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_rows_are_checked_by_every_call(lib, kw, code):
    r = rows(**kw)
    assert logprobs(lib, r) == code
    assert backward(lib, r, ldd=1 << 25) == code
    assert route(lib, r) == code


def test_logprobs_arguments(lib):
    assert logprobs(lib, Z=0) == BAD
    assert lib.gmm_logprobs(None, P(16), P(0), 0, P(0), P(16), P(16), P(0), P(0), P(0),
                            P(0)) == BAD
    assert logprobs(lib, Z=18) == UNSUP  # not aligned to a float
    assert logprobs(lib, rows(dtype=G.GMM_BF16), Z=17) == UNSUP
    for m in (-1, 33):
        assert logprobs(lib, m=m) == BAD
    assert logprobs(lib, ids=0) == BAD   # logp without ids
    assert logprobs(lib, logp=0) == BAD  # ids without logp
    assert logprobs(lib, ti=0) == BAD
    assert logprobs(lib, tv=0) == BAD
    assert logprobs(lib, ids=0, logp=0, H=0, lse=0, m=0) == BAD  # nothing asked for


def test_backward_arguments(lib):
    for name in ("Z", "ids", "lse", "H", "ti", "dtop", "dZ"):
        assert backward(lib, **{name: 0}) == BAD, name
    assert backward(lib, m=0, dlogp=0, dH=0, dlse=0) == BAD  # no upstream gradient
    for m in (-1, 33):
        assert backward(lib, m=m) == BAD
    assert backward(lib, ldd=7) == BAD
    assert backward(lib, ldd=(1 << 40) + 1) == UNSUP
    assert backward(lib, dZ=34) == UNSUP
    assert backward(lib, dZ=16, ldd=9) == BAD  # in place needs the same stride


def test_route_arguments(lib):
    for m in (0, 9):
        assert route(lib, m=m) == BAD
    assert route(lib, rows(K=2), m=3) == BAD  # m > K
    for name in ("Z", "idx", "resp"):
        assert route(lib, **{name: 0}) == BAD, name


def test_no_rows_is_no_work(lib):
    r = rows(N=0)
    assert logprobs(lib, r, Z=0, ids=0, logp=0, H=0, lse=0, m=0) == G.GMM_OK
    assert backward(lib, r, Z=0, lse=0, dZ=0) == G.GMM_OK
    assert route(lib, r, Z=0, idx=0, resp=0) == G.GMM_OK
    p = G.gmm_moe_problem(0, 2, 4, 16, 8, G.GMM_BF16, 0, 16, 16)
    assert lib.gmm_moe(ctypes.byref(p), *([P(0)] * 7), 0, P(0)) == G.GMM_OK


def moe_p(T=4, m=2, E=4, D=16, F=8, dtype=G.GMM_BF16, act=0, ldx=16, ldy=16):
    return G.gmm_moe_problem(T, m, E, D, F, dtype, act, ldx, ldy)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(m=0), BAD), (dict(m=9), BAD), (dict(E=0), BAD), (dict(D=0), BAD),
    (dict(F=0), BAD), (dict(dtype=5), BAD), (dict(act=2), BAD), (dict(act=-1), BAD),
    (dict(ldx=8), BAD), (dict(ldy=15), BAD), (dict(dtype=G.GMM_F32), UNSUP), (dict(T=257), UNSUP),
    (dict(E=1025), UNSUP), (dict(D=12), UNSUP), (dict(F=12), UNSUP), (dict(ldx=20), UNSUP),
    (dict(ldx=1 << 39), UNSUP),
    (dict(F=(1 << 20) + 8), UNSUP), (dict(ldy=(1 << 40) + 1), UNSUP),
])
def test_moe_problems(lib, kw, code):
    p, n = moe_p(**kw), ctypes.c_size_t(0)
    assert lib.gmm_moe_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.gmm_moe(ctypes.byref(p), P(16), P(16), P(16), P(16), P(16), P(16), P(256), 1 << 40,
                       P(0)) == code


def test_moe_arguments(lib):
    p, n = moe_p(), ctypes.c_size_t(0)
    assert lib.gmm_moe_workspace_size(None, ctypes.byref(n)) == BAD
    assert lib.gmm_moe_workspace_size(ctypes.byref(p), None) == BAD
    assert lib.gmm_moe_workspace_size(ctypes.byref(p), ctypes.byref(n)) == G.GMM_OK
    assert n.value == 256 + 2 * 256  # T * m * F halves of 2 bytes, each rounded up to 256

    def call(X=16, idx=16, resp=16, Wu=16, Wd=16, Y=16, ws=256, size=n.value):
        return lib.gmm_moe(ctypes.byref(p), P(X), P(idx), P(resp), P(Wu), P(Wd), P(Y), P(ws),
                           size, P(0))

    for name in ("X", "idx", "resp", "Wu", "Wd", "Y"):
        assert call(**{name: 0}) == BAD, name
    for name in ("X", "Wu", "Wd"):
        assert call(**{name: 24}) == UNSUP, name
    assert call(Y=17) == UNSUP
    assert call(ws=0) == WS
    assert call(ws=128) == WS
    assert call(size=n.value - 1) == WS


def test_binding_refuses_what_it_cannot_pass(lib):
    Z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        G.gmm_logprobs(Z)
    with pytest.raises(TypeError):
        G.gmm_logprobs(Z.double())
    with pytest.raises(ValueError):
        G.gmm_logprobs(Z.t())
    with pytest.raises(ValueError):
        G.gmm_logprobs(Z[0])
    with pytest.raises(TypeError):
        G.gmm_route(Z.int(), 2)
    with pytest.raises(ValueError):
        G.gmm_logprobs_backward(Z, None, torch.zeros(4), dtop=torch.zeros(4, 2))
    with pytest.raises(ValueError):
        G.gmm_moe(Z, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), Z, Z)


def test_a_scale_beyond_its_range_is_refused(lib):
    """scale * log2 e has to be finite: the exponents are formed with it."""
    r = rows(scale=2.5e38)
    assert logprobs(lib, r) == UNSUP
    assert backward(lib, r) == UNSUP
    assert route(lib, r) == UNSUP
