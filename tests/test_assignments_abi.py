"""The calls around a vocabulary and a router refuse bad arguments on the host, before anything is
enqueued (no GPU needed), and the binding refuses tensors it cannot pass on."""
import ctypes

import pytest
import torch

from soft_clustering_em_b200 import gmm as G

P = ctypes.c_void_p
BAD, UNSUP, WS, OK = (G.GMM_ERR_INVALID_ARG, G.GMM_ERR_UNSUPPORTED, G.GMM_ERR_WORKSPACE, G.GMM_OK)


@pytest.fixture(scope="module")
def lib():
    from soft_clustering_em_b200 import build

    build.build()
    return G.load_library()


def rows(N=12, ld=8, K=8, dtype=G.GMM_F32, scale=1.0):
    return ctypes.byref(G.gmm_rows(N, ld, K, dtype, scale))


def loss(lib, r=None, Z=16, idx=16, m=2, mask=0, off=0, S=1, out=(16,) * 5, ws=256, size=1 << 40):
    return lib.gmm_route_loss(r or rows(), P(Z), P(idx), m, P(mask), P(off), S, *map(P, out), P(0),
                              P(ws), size, P(0))


def grad(lib, r=None, Z=16, idx=16, m=2, dresp=16, renorm=0, counts=16, n=16, db=16, dz=16, mask=0,
         off=0, S=1, dZ=32, ldd=8):
    return lib.gmm_route_backward(r or rows(), P(Z), P(idx), m, P(dresp), renorm, P(counts), P(n),
                                  P(db), P(dz), P(mask), P(off), S, P(dZ), ldd, P(0), P(0))


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(K=0), BAD), (dict(ld=7), BAD), (dict(dtype=3), BAD),
    (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=2.5e38), UNSUP),
    (dict(K=1025, ld=2000), UNSUP), (dict(N=1 << 30), UNSUP), (dict(ld=(1 << 40) + 1), UNSUP),
])
def test_router_rows(lib, kw, code):
    assert loss(lib, rows(**kw)) == code
    assert grad(lib, rows(**kw), ldd=2000) == code


def test_router_loss_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.gmm_route_loss_workspace_size(rows(), 1, None) == BAD
    assert lib.gmm_route_loss_workspace_size(None, 1, ctypes.byref(n)) == BAD
    assert lib.gmm_route_loss_workspace_size(rows(), -1, ctypes.byref(n)) == BAD
    assert lib.gmm_route_loss_workspace_size(rows(), (1 << 20) + 1, ctypes.byref(n)) == UNSUP
    assert lib.gmm_route_loss_workspace_size(rows(), 1, ctypes.byref(n)) == OK
    assert loss(lib, Z=0) == BAD
    assert loss(lib, idx=0) == BAD
    assert loss(lib, Z=18) == UNSUP
    assert loss(lib, out=(0,) * 5) == BAD
    for m in (0, 9):
        assert loss(lib, m=m) == BAD
    assert loss(lib, S=2) == BAD  # two segments need offsets
    assert loss(lib, ws=0) == WS
    assert loss(lib, ws=128) == WS
    assert loss(lib, size=n.value - 1) == WS
    assert loss(lib, off=16, S=0) == OK  # no segment is no work


def test_router_gradient_arguments(lib):
    assert grad(lib, dresp=0, db=0, dz=0) == BAD  # no upstream gradient
    for name in ("Z", "idx", "counts", "n", "dZ"):
        assert grad(lib, **{name: 0}) == BAD, name
    for m in (0, 9):
        assert grad(lib, m=m) == BAD
    assert grad(lib, S=2) == BAD
    assert grad(lib, off=16, S=0) == BAD
    assert grad(lib, ldd=7) == BAD
    assert grad(lib, dZ=16, ldd=9) == BAD  # in place needs the same stride
    assert grad(lib, dZ=34) == UNSUP
    assert grad(lib, Z=18) == UNSUP
    assert grad(lib, ldd=(1 << 40) + 1) == UNSUP
    assert grad(lib, rows(N=0), Z=0, idx=0, dZ=0) == OK


def test_a_scale_is_a_number():
    import fractions

    import numpy as np

    Z = torch.zeros(3, 8)
    for half in (0.5, np.float32(0.5), np.float64(0.5), np.array(0.5), fractions.Fraction(1, 2),
                 torch.tensor(0.5)):
        assert G._rows(Z, half).scale == 0.5
    assert G._rows(Z, 2).scale == 2.0
    for bad in ("0.5", b"0.5", None, [0.5], 0.5j):
        with pytest.raises(TypeError):
            G._rows(Z, bad)


def problem(N=4, m=2, K=6, D=8, dtype=G.GMM_BF16, scale=1.0, ldw=8, ldy=8):
    return ctypes.byref(G.gmm_embed_problem(N, m, K, D, dtype, scale, ldw, ldy))


def embed(lib, p=None, W=16, idx=16, resp=0, Y=16):
    return lib.gmm_embed(p or problem(), P(W), P(idx), P(resp), P(Y), P(0), P(0))


def embed_grad(lib, p=None, dY=16, idx=16, resp=16, W=16, dW=16, t=G.GMM_F32, ldd=8, dresp=16,
               ws=256, size=1 << 40):
    return lib.gmm_embed_backward(p or problem(), P(dY), P(idx), P(resp), P(W), P(dW), t, ldd, 0,
                                  P(dresp), P(0), P(ws), size, P(0))


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(m=0), BAD), (dict(m=9), BAD), (dict(K=0), BAD), (dict(D=0), BAD),
    (dict(dtype=3), BAD), (dict(scale=float("inf")), BAD), (dict(ldw=7), BAD), (dict(ldy=7), BAD),
    (dict(K=(1 << 24) + 1), UNSUP), (dict(D=(1 << 20) + 1, ldw=1 << 21, ldy=1 << 21), UNSUP),
    (dict(N=1 << 30), UNSUP), (dict(N=1 << 21, D=1 << 20, ldw=1 << 20, ldy=1 << 20), UNSUP),
    (dict(ldw=(1 << 40) + 1), UNSUP), (dict(ldy=(1 << 40) + 1), UNSUP),
])
def test_embed_problems(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert embed(lib, problem(**kw)) == code
    assert embed_grad(lib, problem(**kw), ldd=1 << 21) == code
    assert lib.gmm_embed_workspace_size(problem(**kw), ctypes.byref(n)) == code


def test_embed_arguments(lib):
    for name in ("W", "idx", "Y"):
        assert embed(lib, **{name: 0}) == BAD, name
    for name in ("W", "Y"):
        assert embed(lib, **{name: 17}) == UNSUP, name
    assert embed(lib, problem(N=0), W=0, idx=0, Y=0) == OK


def test_embed_gradient_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.gmm_embed_workspace_size(problem(), None) == BAD
    assert lib.gmm_embed_workspace_size(problem(), ctypes.byref(n)) == OK
    assert embed_grad(lib, dW=0, dresp=0) == BAD
    for name in ("dY", "idx", "W"):
        assert embed_grad(lib, **{name: 0}) == BAD, name
    assert embed_grad(lib, t=G.GMM_F16) == BAD  # the rows' type or float32
    assert embed_grad(lib, ldd=7) == BAD
    assert embed_grad(lib, ldd=(1 << 40) + 1) == UNSUP
    for name in ("dY", "W"):
        assert embed_grad(lib, **{name: 17}) == UNSUP, name
    assert embed_grad(lib, dW=18) == UNSUP
    assert embed_grad(lib, ws=0) == WS
    assert embed_grad(lib, ws=264) == WS
    assert embed_grad(lib, size=n.value - 1) == WS


def select(lib, r=None, Z=16, w=4, scores=16, ended=0, end_id=0, m=4, out=(16, 16, 16), ws=256,
           size=1 << 40):
    return lib.gmm_beam_select(r or rows(), P(Z), w, P(scores), P(ended), end_id, m, *map(P, out),
                               P(0), P(ws), size, P(0))


def test_selection_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.gmm_beam_workspace_size(rows(), 4, 4, None) == BAD
    assert lib.gmm_beam_workspace_size(rows(), 4, 4, ctypes.byref(n)) == OK
    for kw, code in ((dict(K=0), BAD), (dict(ld=7), BAD), (dict(dtype=7), BAD),
                     (dict(scale=-1.0), BAD), (dict(K=(1 << 24) + 1, ld=1 << 25), UNSUP),
                     (dict(N=1 << 31), UNSUP)):
        assert select(lib, rows(**kw)) == code, kw
    for w in (0, 33, 5):  # 5 does not divide the 12 rows
        assert select(lib, w=w) == BAD
    for m in (0, 33):
        assert select(lib, m=m) == BAD
    assert select(lib, Z=0) == BAD
    assert select(lib, Z=18) == UNSUP
    assert select(lib, scores=0) == BAD
    for i in range(3):
        assert select(lib, out=tuple(0 if i == j else 16 for j in range(3))) == BAD
    for end in (-1, 8):
        assert select(lib, ended=16, end_id=end) == BAD
    assert select(lib, ws=0) == WS
    assert select(lib, ws=128) == WS
    assert select(lib, size=n.value - 1) == WS
    assert select(lib, rows(N=0), Z=0, scores=0, out=(0, 0, 0), ws=0, size=0) == OK


def state(base=16, row=64, outer=2, outer_stride=32, count=4, pos=8, by_len=1):
    return G.gmm_beam_state(base, row, outer, outer_stride, count, pos, by_len)


def reorder(lib, B=2, w=2, parent=16, lens=0, n=1, st=None, **kw):
    st = state(**kw) if st is None else st
    return lib.gmm_beam_reorder(B, w, P(parent), P(lens), n, ctypes.byref(st), P(0), P(0))


def test_reordering_arguments(lib):
    assert reorder(lib, parent=0) == BAD
    for w in (0, 33):
        assert reorder(lib, w=w) == BAD
    assert reorder(lib, B=-1) == BAD
    assert reorder(lib, n=-1) == BAD
    assert reorder(lib, B=1 << 31) == UNSUP
    for name in ("row", "outer", "outer_stride", "count", "pos"):
        assert reorder(lib, **{name: -1}) == BAD, name
    assert reorder(lib, base=0) == BAD
    assert reorder(lib, row=0) == BAD           # the beams' rows are the same
    assert reorder(lib, outer_stride=31) == BAD  # pieces overlap
    assert reorder(lib, row=1 << 36, outer=1, count=1 << 30, pos=1 << 6) == UNSUP  # 2^32 columns
    assert reorder(lib, row=1 << 41, outer=1, count=1 << 31, pos=16) == UNSUP
    assert lib.gmm_beam_reorder(1, 2, P(16), P(0), 1, None, P(0), P(0)) == BAD
    assert reorder(lib, B=0, parent=0) == OK
    assert reorder(lib, n=0, parent=0) == OK


def test_a_state_named_twice(lib):
    for second in (state(), state(outer=1), state(pos=4)):
        two = (type(second) * 2)(state(), second)
        assert lib.gmm_beam_reorder(3, 2, P(16), P(0), 2, two, P(0), P(0)) == BAD
    two = (type(second) * 2)(state(count=0), state(count=0))  # nothing in them
    assert lib.gmm_beam_reorder(3, 2, P(16), P(0), 2, two, P(0), P(0)) == OK


def test_the_binding_packs_states_as_the_header_does():
    st = state()
    packed = G._STATE.pack(16, 64, 2, 32, 4, 8, 1)
    assert len(packed) == ctypes.sizeof(st) and bytes(st)[:52] == packed[:52]


def layout(t, rows, dim):
    return G._state_layout(t.shape, t.stride(), t.element_size(), rows, dim)


def test_states_that_can_be_reordered():
    t = torch.zeros(6, 3, 5, 4)
    assert layout(t, 6, 2) == (240, 3, 80, 5, 16, 1)
    assert layout(t, 6, 1) == (240, 1, 0, 3, 80, 1)
    assert layout(t, 6, None) == (240, 1, 0, 1, 240, 0)
    layers = torch.zeros(2, 6, 3, 5, 4)[1]
    assert layout(layers, 6, 2) == (240, 3, 80, 5, 16, 1)
    with pytest.raises(ValueError):
        layout(t.transpose(2, 3), 6, 2)  # positions' widths do not lie densely
    with pytest.raises(ValueError):
        layout(t, 5, 2)
    by_position = torch.zeros(5, 6, 4).transpose(0, 1)  # positions first
    with pytest.raises(ValueError):
        layout(by_position, 6, 1)


def test_binding_refuses_what_it_cannot_pass(lib):
    Z, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        G.gmm_route_loss(Z, idx)
    with pytest.raises(ValueError, match="CUDA"):
        G.gmm_embed(Z, idx)
    with pytest.raises(ValueError, match="CUDA"):
        G.gmm_embed_backward(Z, idx, 8)
    with pytest.raises(ValueError, match="CUDA"):
        G.gmm_beam_select(Z, torch.zeros(2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        G.gmm_beam_reorder(Z, torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        G.gmm_route_loss(Z.double(), idx)
    with pytest.raises(TypeError):
        G._segments(Z, idx.long(), None, None)
    with pytest.raises(TypeError):
        G._segments(Z, idx, torch.zeros(4), None)
    with pytest.raises(ValueError):
        G._segments(Z, idx, torch.zeros(5, dtype=torch.bool), None)
    with pytest.raises(ValueError):
        G._segments(Z, idx, None, torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError):
        G._choices(idx, None, 5)
    with pytest.raises(TypeError):
        G._choices(idx, torch.zeros(4, 2, dtype=torch.float64), 4)
    with pytest.raises(ValueError):
        G._ld(Z.t(), "W")
