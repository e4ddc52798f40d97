"""Thin Python binding of the C ABI in include/gmm.h (argument marshalling only).

Every entry point keeps its C name.  Arrays are torch CUDA tensors; the binding
passes their device pointers and the current CUDA stream to the library and
does no arithmetic of its own.  The library must be built
(``python -m soft_clustering_em_b200.build``); if it is missing every call
raises -- there is no fallback implementation.
"""
import ctypes
import functools
import math
import os
import struct
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libscem_gmm.so")

GMM_OK, GMM_ERR_INVALID_ARG, GMM_ERR_UNSUPPORTED, GMM_ERR_CUDA = 0, 1, 2, 3
GMM_ERR_NUMERIC, GMM_ERR_TIMEOUT, GMM_ERR_WORKSPACE = 4, 5, 6
GMM_F32, GMM_BF16, GMM_F16 = 0, 1, 2
GMM_ACT_SILU, GMM_ACT_GELU = 0, 1
GMM_INIT_VAR_ONE, GMM_INIT_VAR_DATA = 0, 1
GMM_DEVFLAG_NONFINITE_X, GMM_DEVFLAG_BAD_PARAMS, GMM_DEVFLAG_WAIT_TIMEOUT = 0x1, 0x2, 0x4
GMM_DEVFLAG_X_RANGE, GMM_DEVFLAG_BAD_INDEX = 0x8, 0x10

EXPORTS = ("gmm_workspace_size", "gmm_plan", "gmm_init", "gmm_init_rows", "gmm_em_step",
           "gmm_em_step_hard", "gmm_em_step_spherical", "gmm_kmeans_step", "gmm_em_step_noalloc",
           "gmm_host_staging_size", "gmm_em_step_host",
           "gmm_estep_stats", "gmm_mstep", "gmm_fit", "gmm_loglik",
           "gmm_assign_topm", "gmm_ivf_workspace_size", "gmm_ivf_build", "gmm_logprobs",
           "gmm_logprobs_backward", "gmm_route", "gmm_moe_workspace_size", "gmm_moe",
           "gmm_route_loss_workspace_size", "gmm_route_loss", "gmm_route_backward", "gmm_embed",
           "gmm_embed_workspace_size", "gmm_embed_backward", "gmm_beam_workspace_size",
           "gmm_beam_select", "gmm_beam_reorder",
           "gmm_device_status",
           "gmm_trace_fused", "gmm_set_wait_budget", "gmm_launch_count", "gmm_status_string")


class gmm_problem(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("D", ctypes.c_int32), ("K", ctypes.c_int32),
                ("xdtype", ctypes.c_int32), ("var_floor", ctypes.c_float)]


class gmm_plan_info(ctypes.Structure):
    _fields_ = [("tensor_cores", ctypes.c_int32), ("cluster_ctas", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("fit_one_launch", ctypes.c_int32),
                ("chunk_rows", ctypes.c_int64)]


class gmm_rows(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("ld", ctypes.c_int64), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class gmm_moe_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("m", ctypes.c_int32), ("E", ctypes.c_int32),
                ("D", ctypes.c_int32), ("F", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class gmm_embed_problem(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("m", ctypes.c_int32), ("K", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("ldw", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class gmm_beam_state(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("outer", ctypes.c_int64), ("outer_stride", ctypes.c_int64),
                ("count", ctypes.c_int64), ("pos_bytes", ctypes.c_int64),
                ("by_len", ctypes.c_int32)]


class GmmError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library and declare its signatures (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is not built; run "
                           "`python -m soft_clustering_em_b200.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    PP = ctypes.POINTER(gmm_problem)
    lib.gmm_workspace_size.argtypes = [PP, ctypes.POINTER(SZ)]
    lib.gmm_plan.argtypes = [PP, ctypes.POINTER(gmm_plan_info)]
    lib.gmm_init.argtypes = [PP, P, ctypes.c_uint64, I32, P, P, P, P, SZ, P]
    lib.gmm_init_rows.argtypes = [PP, P, ctypes.POINTER(I64), I32, P, P, P, P, SZ, P]
    lib.gmm_em_step.argtypes = [PP, P, P, P, P, P, P, SZ, P]
    lib.gmm_em_step_noalloc.argtypes = [PP, P, P, P, P, P, P, P]
    lib.gmm_em_step_hard.argtypes = [PP, P, P, P, P, P, P, P, SZ, P]
    lib.gmm_em_step_spherical.argtypes = [PP, P, P, P, P, P, P, SZ, P]
    lib.gmm_kmeans_step.argtypes = [PP, P, P, P, P, P, SZ, P]
    lib.gmm_host_staging_size.argtypes = [PP, I64, ctypes.POINTER(SZ)]
    lib.gmm_em_step_host.argtypes = [PP, P, I64, P, SZ, P, P, P, P, P, SZ, P, P]
    lib.gmm_estep_stats.argtypes = [PP, P, P, P, P, P, P, SZ, P]
    lib.gmm_mstep.argtypes = [PP, P, I32, P, P, P, P, P]
    lib.gmm_fit.argtypes = [PP, P, I32, P, P, P, P, P, SZ, P]
    lib.gmm_loglik.argtypes = [PP, P, P, P, P, P, P, SZ, P]
    lib.gmm_assign_topm.argtypes = [PP, P, P, P, P, I32, P, P, P, SZ, P]
    lib.gmm_ivf_workspace_size.argtypes = [I64, I32, ctypes.POINTER(SZ)]
    lib.gmm_ivf_build.argtypes = [I64, I32, I32, P, P, ctypes.c_float, P, P, I64, P, SZ, P]
    PR, PM = ctypes.POINTER(gmm_rows), ctypes.POINTER(gmm_moe_problem)
    lib.gmm_logprobs.argtypes = [PR, P, P, I32, P, P, P, P, P, P, P]
    lib.gmm_logprobs_backward.argtypes = [PR, P, P, P, P, P, P, P, I32, P, P, P, I64, P, P]
    lib.gmm_route.argtypes = [PR, P, I32, I32, P, P, P, P]
    lib.gmm_moe_workspace_size.argtypes = [PM, ctypes.POINTER(SZ)]
    lib.gmm_moe.argtypes = [PM, P, P, P, P, P, P, P, SZ, P]
    PE = ctypes.POINTER(gmm_embed_problem)
    lib.gmm_route_loss_workspace_size.argtypes = [PR, I32, ctypes.POINTER(SZ)]
    lib.gmm_route_loss.argtypes = [PR, P, P, I32, P, P, I32, P, P, P, P, P, P, P, SZ, P]
    lib.gmm_route_backward.argtypes = [PR, P, P, I32, P, I32, P, P, P, P, P, P, I32, P, I64, P, P]
    lib.gmm_embed.argtypes = [PE, P, P, P, P, P, P]
    lib.gmm_embed_workspace_size.argtypes = [PE, ctypes.POINTER(SZ)]
    lib.gmm_embed_backward.argtypes = [PE, P, P, P, P, P, I32, I64, I32, P, P, P, SZ, P]
    lib.gmm_beam_workspace_size.argtypes = [PR, I32, I32, ctypes.POINTER(SZ)]
    lib.gmm_beam_select.argtypes = [PR, P, I32, P, P, I32, I32, P, P, P, P, P, SZ, P]
    lib.gmm_beam_reorder.argtypes = [I64, I32, P, P, I32, P, P, P]
    lib.gmm_device_status.argtypes = [P, SZ, P, ctypes.POINTER(ctypes.c_uint32), I32]
    lib.gmm_trace_fused.argtypes = [P, P]
    lib.gmm_set_wait_budget.argtypes = [ctypes.c_uint64]
    lib.gmm_launch_count.argtypes = [ctypes.POINTER(ctypes.c_uint64)]
    lib.gmm_status_string.argtypes = [ctypes.c_int]
    lib.gmm_status_string.restype = ctypes.c_char_p
    for name in EXPORTS[:-1]:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(s: int) -> str:
    return load_library().gmm_status_string(int(s)).decode()


def _check(rc, what):
    if rc != GMM_OK:
        raise GmmError(rc, what)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def xdtype_of(X) -> int:
    if X.dtype == torch.float32:
        return GMM_F32
    if X.dtype == torch.bfloat16:
        return GMM_BF16
    raise TypeError(f"X must be float32 or bfloat16, got {X.dtype}")


def problem(N, D, K, xdtype=GMM_F32, var_floor=1e-6) -> gmm_problem:
    return gmm_problem(int(N), int(D), int(K), int(xdtype), float(var_floor))


def problem_for(X, K, var_floor=1e-6) -> gmm_problem:
    N, D = X.shape
    return problem(N, D, K, xdtype_of(X), var_floor)


def gmm_workspace_size(p: gmm_problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().gmm_workspace_size(ctypes.byref(p), ctypes.byref(n)),
           "gmm_workspace_size")
    return int(n.value)


def gmm_plan(p: gmm_problem) -> dict:
    """How the library runs problem p on the current device."""
    info = gmm_plan_info()
    _check(load_library().gmm_plan(ctypes.byref(p), ctypes.byref(info)), "gmm_plan")
    return {f: int(getattr(info, f)) for f, _ in gmm_plan_info._fields_}


def workspace(p: gmm_problem, device=None) -> torch.Tensor:
    """A zero-filled device workspace for problem p (caller-owned, reusable)."""
    return torch.zeros(gmm_workspace_size(p), dtype=torch.uint8, device=device or "cuda")


def _ws(p, ws, device):
    return workspace(p, device) if ws is None else ws


def _init_out(X, K):
    w = torch.empty(K, dtype=torch.float32, device=X.device)
    mu = torch.empty(K, X.shape[1], dtype=torch.float32, device=X.device)
    return w, mu, torch.empty_like(mu)


def gmm_init(X, seed, K, init_var=GMM_INIT_VAR_DATA, var_floor=1e-6, ws=None, stream=None):
    """Initial (w, mu, var): means at K distinct rows of X chosen from `seed`."""
    p = problem_for(X, K, var_floor)
    ws = _ws(p, ws, X.device)
    w, mu, var = _init_out(X, K)
    _check(load_library().gmm_init(ctypes.byref(p), _ptr(X), int(seed) & ((1 << 64) - 1),
                                   int(init_var), _ptr(w), _ptr(mu), _ptr(var), _ptr(ws),
                                   ws.numel(), _stream(stream)), "gmm_init")
    return w, mu, var


def gmm_init_rows(X, rows, K, init_var=GMM_INIT_VAR_DATA, var_floor=1e-6, ws=None, stream=None):
    """Initial (w, mu, var) from the K chosen rows of X (host int64 indices)."""
    p = problem_for(X, K, var_floor)
    ws = _ws(p, ws, X.device)
    rows = (ctypes.c_int64 * K)(*[int(r) for r in rows])
    w, mu, var = _init_out(X, K)
    _check(load_library().gmm_init_rows(ctypes.byref(p), _ptr(X), rows, int(init_var), _ptr(w),
                                        _ptr(mu), _ptr(var), _ptr(ws), ws.numel(),
                                        _stream(stream)), "gmm_init_rows")
    return w, mu, var


def gmm_em_step(X, w, mu, var, loglik=None, var_floor=1e-6, ws=None, stream=None):
    """One fused EM iteration in place; loglik (1 double, device) gets LL of the input."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    _check(load_library().gmm_em_step(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu), _ptr(var),
                                      _ptr(loglik), _ptr(ws), ws.numel(), _stream(stream)),
           "gmm_em_step")


def gmm_em_step_hard(X, w, mu, var, labels=None, loglik=None, var_floor=1e-6, ws=None,
                     stream=None):
    """One classification-EM step in place; labels (N int32) and loglik optional outputs."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    _check(load_library().gmm_em_step_hard(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu),
                                           _ptr(var), _ptr(labels), _ptr(loglik), _ptr(ws),
                                           ws.numel(), _stream(stream)), "gmm_em_step_hard")


def gmm_em_step_spherical(X, w, mu, s2, loglik=None, var_floor=1e-6, ws=None, stream=None):
    """One soft EM step in place with covariances s2_k * I (s2: K floats)."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    _check(load_library().gmm_em_step_spherical(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu),
                                                _ptr(s2), _ptr(loglik), _ptr(ws), ws.numel(),
                                                _stream(stream)), "gmm_em_step_spherical")


def gmm_kmeans_step(X, centers, labels=None, inertia=None, ws=None, stream=None):
    """One Lloyd step in place on centers (K x D); optional labels (N int32) and inertia."""
    p = problem_for(X, centers.shape[0])
    ws = _ws(p, ws, X.device)
    _check(load_library().gmm_kmeans_step(ctypes.byref(p), _ptr(X), _ptr(centers), _ptr(labels),
                                          _ptr(inertia), _ptr(ws), ws.numel(), _stream(stream)),
           "gmm_kmeans_step")


_copy_streams = {}


def copy_stream_for(device):
    """A side stream per device for gmm_em_step_host's host-to-device copies."""
    key = torch.device(device).index if torch.device(device).index is not None else \
        torch.cuda.current_device()
    if key not in _copy_streams:
        _copy_streams[key] = torch.cuda.Stream(device=key)
    return _copy_streams[key]


def gmm_host_staging_size(p: gmm_problem, chunk_rows) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().gmm_host_staging_size(ctypes.byref(p), int(chunk_rows),
                                                ctypes.byref(n)), "gmm_host_staging_size")
    return int(n.value)


def gmm_em_step_host(X_host, w, mu, var, loglik=None, chunk_rows=1 << 18, var_floor=1e-6,
                     staging=None, ws=None, stream=None, copy_stream=None):
    """One EM iteration in place with X in host memory (pinned for overlap).

    X_host: contiguous CPU tensor, float32 or bfloat16, N x D.  The rows are
    copied chunk_rows at a time through device staging on copy_stream (default:
    a side stream of the parameters' device) while the E-step runs on stream.
    """
    if X_host.is_cuda or not X_host.is_contiguous():
        raise ValueError("X_host must be a contiguous host tensor")
    p = problem_for(X_host, w.numel(), var_floor)
    ws = _ws(p, ws, w.device)
    if staging is None:
        staging = torch.empty(gmm_host_staging_size(p, chunk_rows), dtype=torch.uint8,
                              device=w.device)
    cs = copy_stream_for(w.device) if copy_stream is None else copy_stream
    _check(load_library().gmm_em_step_host(ctypes.byref(p), ctypes.c_void_p(X_host.data_ptr()),
                                           int(chunk_rows), _ptr(staging), staging.numel(),
                                           _ptr(w), _ptr(mu), _ptr(var), _ptr(loglik), _ptr(ws),
                                           ws.numel(), _stream(stream), _stream(cs)),
           "gmm_em_step_host")


def stats_size(K, D) -> int:
    """Doubles in a statistics buffer: [N_k (K) | A (K x D) | B (K x D) | LL]."""
    return int(K) * (2 * int(D) + 1) + 1


def gmm_estep_stats(X, w, mu, var, stats=None, var_floor=1e-6, ws=None, stream=None):
    """E-step statistics of the rows of X (fp64 device tensor [N_k | A | B | LL])."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    if stats is None:
        stats = torch.empty(stats_size(w.numel(), X.shape[1]), dtype=torch.float64,
                            device=X.device)
    _check(load_library().gmm_estep_stats(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu), _ptr(var),
                                          _ptr(stats), _ptr(ws), ws.numel(), _stream(stream)),
           "gmm_estep_stats")
    return stats


def gmm_mstep(stats, N_total, w, mu, var, loglik=None, var_floor=1e-6, xdtype=GMM_F32,
              stream=None):
    """M-step in place from the statistics of row shards holding N_total points.

    stats: fp64 device tensor of shape (S,) or (nshards, S), S = stats_size(K, D);
    the shards are summed in order inside the library."""
    K, D = mu.shape
    nshards = 1 if stats.dim() == 1 else stats.shape[0]
    p = problem(N_total, D, K, xdtype, var_floor)
    _check(load_library().gmm_mstep(ctypes.byref(p), _ptr(stats.contiguous()), int(nshards),
                                    _ptr(w), _ptr(mu), _ptr(var), _ptr(loglik), _stream(stream)),
           "gmm_mstep")


def gmm_em_step_noalloc(X, w, mu, var, loglik=None, dev_flags=None, var_floor=1e-6,
                        stream=None):
    """gmm_em_step on the library's built-in scratch: no workspace, no device allocation.

    For callers that may not obtain device memory (see include/gmm.h).  dev_flags
    (1 int32 device tensor, optional) receives the call's device status bits.
    """
    p = problem_for(X, w.numel(), var_floor)
    _check(load_library().gmm_em_step_noalloc(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu),
                                              _ptr(var), _ptr(loglik), _ptr(dev_flags),
                                              _stream(stream)), "gmm_em_step_noalloc")


def gmm_fit(X, w, mu, var, iters, var_floor=1e-6, ws=None, stream=None):
    """iters EM iterations in place; returns the device LL history (iters doubles)."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    ll = torch.zeros(max(int(iters), 1), dtype=torch.float64, device=X.device)
    _check(load_library().gmm_fit(ctypes.byref(p), _ptr(X), int(iters), _ptr(w), _ptr(mu),
                                  _ptr(var), _ptr(ll), _ptr(ws), ws.numel(), _stream(stream)),
           "gmm_fit")
    return ll[:iters]


def gmm_loglik(X, w, mu, var, var_floor=1e-6, ws=None, stream=None):
    """LL of the given parameters as a 1-element device double tensor."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    ll = torch.zeros(1, dtype=torch.float64, device=X.device)
    _check(load_library().gmm_loglik(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu), _ptr(var),
                                     _ptr(ll), _ptr(ws), ws.numel(), _stream(stream)),
           "gmm_loglik")
    return ll


def gmm_assign_topm(X, w, mu, var, m, var_floor=1e-6, ws=None, stream=None):
    """(idx N x m int32, resp N x m float32): the m most responsible components per point."""
    p = problem_for(X, w.numel(), var_floor)
    ws = _ws(p, ws, X.device)
    N = X.shape[0]
    idx = torch.empty(N, int(m), dtype=torch.int32, device=X.device)
    resp = torch.empty(N, int(m), dtype=torch.float32, device=X.device)
    _check(load_library().gmm_assign_topm(ctypes.byref(p), _ptr(X), _ptr(w), _ptr(mu), _ptr(var),
                                          int(m), _ptr(idx), _ptr(resp), _ptr(ws), ws.numel(),
                                          _stream(stream)), "gmm_assign_topm")
    return idx, resp


def gmm_ivf_workspace_size(N, K) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().gmm_ivf_workspace_size(int(N), int(K), ctypes.byref(n)),
           "gmm_ivf_workspace_size")
    return int(n.value)


def gmm_ivf_build(idx, resp, K, tau, ws=None, stream=None):
    """(offsets (K+1) int64, ids (N*m) int64): IVF lists from a top-m assignment.

    idx (N x m int32) and resp (N x m float32) as gmm_assign_topm returns them.
    List k is ids[offsets[k]:offsets[k+1]]; entries past offsets[K] are unused.
    ws: a zeroed uint8 device tensor of gmm_ivf_workspace_size(N, K) bytes
    (allocated here when None); its first word is the device status word.
    """
    if idx.dtype != torch.int32 or resp.dtype != torch.float32:
        raise TypeError("idx must be int32 and resp float32")
    if idx.dim() != 2 or resp.shape != idx.shape or not (idx.is_contiguous()
                                                       and resp.is_contiguous()):
        raise ValueError("idx and resp must be contiguous N x m tensors of the same shape")
    N, m = idx.shape
    if ws is None:
        ws = torch.zeros(gmm_ivf_workspace_size(N, K), dtype=torch.uint8, device=idx.device)
    offsets = torch.empty(int(K) + 1, dtype=torch.int64, device=idx.device)
    ids = torch.empty(N * m, dtype=torch.int64, device=idx.device)
    _check(load_library().gmm_ivf_build(int(N), int(K), int(m), _ptr(idx), _ptr(resp),
                                        float(tau), _ptr(offsets), _ptr(ids), N * m, _ptr(ws),
                                        ws.numel(), _stream(stream)), "gmm_ivf_build")
    return offsets, ids


_DTYPES = {torch.float32: GMM_F32, torch.bfloat16: GMM_BF16, torch.float16: GMM_F16}


# Descriptions by their values (never changed): building one costs more than looking it up.
@functools.lru_cache(maxsize=4096)
def _rows_of(*fields) -> gmm_rows:
    return gmm_rows(*fields)


@functools.lru_cache(maxsize=4096)
def _embed_of(*fields) -> gmm_embed_problem:
    return gmm_embed_problem(*fields)


def _number(x) -> float:
    return math.ldexp(x, 0)  # (float() would take text as well)


def _rows(Z, scale) -> gmm_rows:
    """The rows of a logits tensor (N x K, any row stride, unit column stride)."""
    if Z.dtype not in _DTYPES:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {Z.dtype}")
    if Z.dim() != 2 or (Z.shape[1] > 1 and Z.stride(1) != 1):
        raise ValueError("logits must be N x K with a unit column stride")
    N, K = Z.shape
    ld = Z.stride(0) if N > 1 else max(Z.stride(0), K)
    return _rows_of(N, ld, K, _DTYPES[Z.dtype], _number(scale))


def _same_device(X, *others):
    """Every tensor of a call is on X's CUDA device."""
    if not X.is_cuda:
        raise ValueError("the tensors must be on a CUDA device")
    index = X.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"the tensors are on different devices: {X.device}, {t.device}")


def _vector(t, n, dtype, name):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {n}, got {tuple(t.shape)}")


def _address(t):
    return None if t is None else t.data_ptr()


def _on(stream, X):
    """The context of a call on `stream`: what the call allocates belongs to that stream."""
    if stream.device != X.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {X.device}")
    return torch.cuda.stream(stream)


def _launch(fn, what, device, *args):
    """Call fn(*args, stream) with `device` current, on its current stream."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _launch(fn, what, device, *args)
    # (the raw handle: building a torch.cuda.Stream object costs as much as a launch)
    rc = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if rc != GMM_OK:
        raise GmmError(rc, what)


class RowLogprobs(NamedTuple):
    """Results of gmm_logprobs; logp is None without ids, the alternatives with m = 0."""

    logp: Optional[torch.Tensor]      # N
    entropy: torch.Tensor             # N
    lse: torch.Tensor                 # N
    top_idx: Optional[torch.Tensor]   # N x m int32
    top_logp: Optional[torch.Tensor]  # N x m


def gmm_logprobs(Z, ids=None, m=0, scale=1.0, dev_flags=None, stream=None) -> RowLogprobs:
    """Log probability of the class ids[n] of each row of logits Z, entropy, log-sum-exp, and
    the m most probable classes with their log probabilities.

    Z: N x K float32, bfloat16 or float16, any row stride; the logits are scale * Z.
    ids: N int32, -1 for rows without a label (logp 0).  m <= 32.  dev_flags (1 int32
    device tensor, optional) collects the device status bits.  stream (None: the current one)
    runs the call and owns the results.
    """
    if stream is not None:
        with _on(stream, Z):
            return gmm_logprobs(Z, ids, m, scale, dev_flags)
    r = _rows(Z, scale)
    N, m = Z.shape[0], int(m)
    _same_device(Z, ids, dev_flags)
    _vector(ids, (N,), torch.int32, "ids")
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    out = torch.empty(3, N, dtype=torch.float32, device=Z.device).unbind(0)
    logp, entropy, lse = out if ids is not None else (None, *out[1:])
    top_idx = top_logp = None
    if m > 0:
        top_idx = torch.empty(N, m, dtype=torch.int32, device=Z.device)
        top_logp = torch.empty(N, m, dtype=torch.float32, device=Z.device)
    _launch(load_library().gmm_logprobs, "gmm_logprobs", Z.device, ctypes.byref(r),
            Z.data_ptr(), _address(ids), m, _address(logp), entropy.data_ptr(), lse.data_ptr(),
            _address(top_idx), _address(top_logp), _address(dev_flags))
    return RowLogprobs(logp, entropy, lse, top_idx, top_logp)


def gmm_logprobs_backward(Z, ids, lse, dlogp=None, entropy=None, dentropy=None, dlse=None,
                          top_idx=None, dtop=None, scale=1.0, out=None, dev_flags=None,
                          stream=None):
    """Gradient with respect to Z of gmm_logprobs(Z, ids, m, scale), for the upstream gradients
    dlogp, dentropy, dlse (N float32 each, None: 0) and dtop (N x m float32, or None).

    lse, entropy and top_idx as gmm_logprobs returned them (entropy only with dentropy, top_idx
    with dtop).  out: N x K of Z's type to write to, Z itself included; allocated when None.
    """
    if stream is not None:
        with _on(stream, Z):
            return gmm_logprobs_backward(Z, ids, lse, dlogp, entropy, dentropy, dlse, top_idx,
                                         dtop, scale, out, dev_flags)
    r = _rows(Z, scale)
    N, K = Z.shape
    m = 0 if dtop is None else (dtop.shape[1] if dtop.dim() == 2 else -1)
    if m < 0 or (dtop is not None and top_idx is None):
        raise ValueError("dtop must be N x m and needs top_idx")
    _same_device(Z, ids, lse, dlogp, entropy, dentropy, dlse, top_idx, dtop, out, dev_flags)
    _vector(ids, (N,), torch.int32, "ids")
    for t, name in ((lse, "lse"), (dlogp, "dlogp"), (entropy, "entropy"),
                    (dentropy, "dentropy"), (dlse, "dlse")):
        _vector(t, (N,), torch.float32, name)
    if m:
        _vector(top_idx, (N, m), torch.int32, "top_idx")
        _vector(dtop, (N, m), torch.float32, "dtop")
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    if out is None:
        out = torch.empty(N, K, dtype=Z.dtype, device=Z.device)
    o = _rows(out, 1.0)
    if out.dtype != Z.dtype or out.shape != Z.shape:
        raise ValueError("out must have the shape and type of Z")
    _launch(load_library().gmm_logprobs_backward, "gmm_logprobs_backward", Z.device,
            ctypes.byref(r), Z.data_ptr(), _address(ids), lse.data_ptr(), _address(entropy),
            _address(dlogp), _address(dentropy), _address(dlse), m,
            _address(top_idx) if m else None, _address(dtop) if m else None, out.data_ptr(), o.ld,
            _address(dev_flags))
    return out


def gmm_route(Z, m, renorm=False, scale=1.0, dev_flags=None, stream=None):
    """(idx N x m int32, resp N x m float32): the m most probable classes of each row of logits
    and their probabilities, divided by their sum with renorm; -1 and 0 where classes run out.
    """
    if stream is not None:
        with _on(stream, Z):
            return gmm_route(Z, m, renorm, scale, dev_flags)
    r = _rows(Z, scale)
    _same_device(Z, dev_flags)
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    N, m = Z.shape[0], int(m)
    idx = torch.empty(N, max(m, 0), dtype=torch.int32, device=Z.device)
    resp = torch.empty(N, max(m, 0), dtype=torch.float32, device=Z.device)
    _launch(load_library().gmm_route, "gmm_route", Z.device, ctypes.byref(r),
            Z.data_ptr(), m, int(bool(renorm)), idx.data_ptr(), resp.data_ptr(),
            _address(dev_flags))
    return idx, resp


def moe_problem(X, idx, W_down, act=GMM_ACT_SILU, out=None) -> gmm_moe_problem:
    """The problem of a gmm_moe call on these tensors."""
    if X.dtype not in _DTYPES:
        raise TypeError(f"X must be bfloat16 or float16, got {X.dtype}")
    T, D = X.shape
    E, _, F = W_down.shape
    ldx, ldy = [D if T <= 1 or t is None else t.stride(0) for t in (X, out)]
    return gmm_moe_problem(T, idx.shape[1], E, D, F, _DTYPES[X.dtype], int(act), ldx, ldy)


def gmm_moe_workspace_size(p: gmm_moe_problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().gmm_moe_workspace_size(ctypes.byref(p), ctypes.byref(n)),
           "gmm_moe_workspace_size")
    return int(n.value)


def gmm_moe(X, idx, resp, W_up, W_down, act=GMM_ACT_SILU, out=None, ws=None, stream=None,
            dev_flags=None):
    """Mixture-of-experts layer for a few tokens: for each token the sum over its choices of
    resp * W_down[e] (act(W_gate[e] x) * (W_lin[e] x)).

    X: T x D bfloat16 or float16 (T <= 256, any row stride that is a multiple of 8); idx, resp:
    T x m as gmm_route or gmm_assign_topm return them, -1 for an unused choice; W_up:
    E x 2F x D, W_gate's F rows over W_lin's; W_down: E x D x F.  Returns T x D of X's type.
    ws: a uint8 device tensor of gmm_moe_workspace_size bytes (allocated here when None), its
    first word the device status word: zero it once to read it with gmm_device_status.
    dev_flags (1 int32 device tensor, optional) collects the device status bits, with or without
    a ws (with one: all that its status word holds).  stream (None: the current one) runs the call
    and owns what is allocated here.
    """
    if stream is not None:
        with _on(stream, X):
            return gmm_moe(X, idx, resp, W_up, W_down, act, out, ws, None, dev_flags)
    if X.dim() != 2 or idx.dim() != 2 or W_up.dim() != 3 or W_down.dim() != 3:
        raise ValueError("X is T x D, idx T x m, W_up E x 2F x D, W_down E x D x F")
    (T, D), (E, _, F) = X.shape, W_down.shape
    _same_device(X, idx, resp, W_up, W_down, out, ws, dev_flags)
    _vector(idx, (T, idx.shape[1]), torch.int32, "idx")
    _vector(resp, (T, idx.shape[1]), torch.float32, "resp")
    _vector(W_up, (E, 2 * F, D), X.dtype, "W_up")
    _vector(W_down, (E, D, F), X.dtype, "W_down")
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    if out is None:
        out = torch.empty(T, D, dtype=X.dtype, device=X.device)
    if out.dtype != X.dtype or out.shape != X.shape:
        raise ValueError("out must have the shape and type of X")
    for t in (X, out):
        if D > 1 and t.stride(1) != 1:
            raise ValueError("X and out must have a unit column stride")
    p = moe_problem(X, idx, W_down, act, out)
    if ws is None:
        ws = torch.empty(gmm_moe_workspace_size(p), dtype=torch.uint8, device=X.device)
        if dev_flags is not None:
            ws[:4].zero_()
    _launch(load_library().gmm_moe, "gmm_moe", X.device, ctypes.byref(p), X.data_ptr(),
            idx.data_ptr(), resp.data_ptr(), W_up.data_ptr(), W_down.data_ptr(), out.data_ptr(),
            ws.data_ptr(), ws.numel())
    if dev_flags is not None:
        dev_flags |= ws[:4].view(torch.int32)
    return out


class RouteLoss(NamedTuple):
    """Results of gmm_route_loss for S segments of rows and K experts."""

    balance: torch.Tensor  # S
    z: torch.Tensor        # S
    load: torch.Tensor     # S x K: mean probabilities
    counts: torch.Tensor   # S x K int32: choices
    rows: torch.Tensor     # S int32: rows that count


def _segments(Z, idx, mask, offsets):
    """Checks of what says which rows count where; returns the number of segments."""
    N = Z.shape[0]
    if idx is not None:
        if idx.dim() != 2:
            raise ValueError("idx must be N x m")
        _vector(idx, (N, idx.shape[1]), torch.int32, "idx")
    if mask is not None:
        _vector(mask, (N,), torch.bool if mask.dtype == torch.bool else torch.uint8, "mask")
    if offsets is None:
        return 1
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be S + 1 row numbers")
    _vector(offsets, offsets.shape, torch.int32, "offsets")
    return offsets.shape[0] - 1


def _bytes(size_fn, what, *args):
    n = ctypes.c_size_t(0)
    _check(size_fn(*args, ctypes.byref(n)), what)
    return int(n.value)


@functools.lru_cache(maxsize=4096)
def _route_loss_bytes(N, K, S):
    return _bytes(load_library().gmm_route_loss_workspace_size, "gmm_route_loss_workspace_size",
                  ctypes.byref(gmm_rows(N, K, K, GMM_F32, 1.0)), S)


@functools.lru_cache(maxsize=4096)
def _embed_bytes(N, m, K, D, dtype):
    return gmm_embed_workspace_size(gmm_embed_problem(N, m, K, D, dtype, 1.0, D, D))


@functools.lru_cache(maxsize=4096)
def _beam_bytes(N, w, m):
    return _bytes(load_library().gmm_beam_workspace_size, "gmm_beam_workspace_size",
                  ctypes.byref(gmm_rows(N, 1, 1, GMM_F32, 1.0)), w, m)


def gmm_route_loss(Z, idx, offsets=None, mask=None, scale=1.0, ws=None, dev_flags=None,
                   stream=None) -> RouteLoss:
    """How the assignment idx loads the experts, the balance loss K sum_k counts_k / (m L) load_k
    (1 for an even load) and the mean squared log-sum-exp z, for each segment of rows.

    Z: N x K router logits (K <= 1024), float32, bfloat16 or float16, any row stride; idx: N x m
    int32 as gmm_route returns it, -1 for an unused choice.  offsets: S + 1 int32, segment s is
    rows offsets[s] to offsets[s + 1]; None: one segment of all rows.  mask: N bool or uint8, 0
    for rows that do not count.  ws: a uint8 device tensor of gmm_route_loss_workspace_size bytes
    (allocated here when None).  dev_flags (1 int32 device tensor, optional) collects the device
    status bits.  stream (None: the current one) runs the call and owns the results.
    """
    if stream is not None:
        with _on(stream, Z):
            return gmm_route_loss(Z, idx, offsets, mask, scale, ws, dev_flags)
    r = _rows(Z, scale)
    _same_device(Z, idx, offsets, mask, ws, dev_flags)
    S = _segments(Z, idx, mask, offsets)
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    N, K = Z.shape
    device = Z.device
    if ws is None:
        ws = torch.empty(_route_loss_bytes(N, K, S), dtype=torch.uint8, device=device)
    balance = torch.empty(S, dtype=torch.float32, device=device)
    z = torch.empty(S, dtype=torch.float32, device=device)
    load = torch.empty(S, K, dtype=torch.float32, device=device)
    counts = torch.empty(S, K, dtype=torch.int32, device=device)
    rows = torch.empty(S, dtype=torch.int32, device=device)
    _launch(load_library().gmm_route_loss, "gmm_route_loss", device, ctypes.byref(r),
            Z.data_ptr(), idx.data_ptr(), idx.shape[1], _address(mask), _address(offsets), S,
            balance.data_ptr(), z.data_ptr(), load.data_ptr(), counts.data_ptr(), rows.data_ptr(),
            _address(dev_flags), ws.data_ptr(), ws.numel())
    return RouteLoss(balance, z, load, counts, rows)


def gmm_route_loss_workspace_size(Z, S=1) -> int:
    """Bytes of gmm_route_loss's workspace for N x K logits like Z and S segments."""
    return _route_loss_bytes(*Z.shape, S)


def gmm_route_backward(Z, idx, dresp=None, renorm=False, counts=None, rows=None, dbalance=None,
                       dz=None, offsets=None, mask=None, scale=1.0, out=None, dev_flags=None,
                       stream=None):
    """Gradient with respect to the router logits Z of gmm_route's weights, for dresp (N x m
    float32, or None), and of gmm_route_loss's losses, for dbalance and dz (S float32, or None).

    idx, renorm, offsets, mask, scale as the forward calls took or gave them; counts and rows as
    gmm_route_loss returned them (with dbalance or dz), or summed over the shards of a batch.
    out: N x K of Z's type to write to, Z itself included; allocated when None.
    """
    if stream is not None:
        with _on(stream, Z):
            return gmm_route_backward(Z, idx, dresp, renorm, counts, rows, dbalance, dz, offsets,
                                      mask, scale, out, dev_flags)
    r = _rows(Z, scale)
    _same_device(Z, idx, dresp, counts, rows, dbalance, dz, offsets, mask, out, dev_flags)
    S = _segments(Z, idx, mask, offsets)
    N, K = Z.shape
    m = idx.shape[1]
    _vector(dresp, (N, m), torch.float32, "dresp")
    _vector(counts, (S, K), torch.int32, "counts")
    _vector(rows, (S,), torch.int32, "rows")
    _vector(dbalance, (S,), torch.float32, "dbalance")
    _vector(dz, (S,), torch.float32, "dz")
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    device = Z.device
    if out is None:
        out, ldd = torch.empty(N, K, dtype=Z.dtype, device=device), K
    else:
        if out.dtype != Z.dtype or out.shape != Z.shape:
            raise ValueError("out must have the shape and type of Z")
        ldd = _ld(out, "out")
    _launch(load_library().gmm_route_backward, "gmm_route_backward", device, ctypes.byref(r),
            Z.data_ptr(), idx.data_ptr(), m, _address(dresp), int(bool(renorm)), _address(counts),
            _address(rows), _address(dbalance), _address(dz), _address(mask), _address(offsets),
            S, out.data_ptr(), ldd, _address(dev_flags))
    return out


def _choices(idx, resp, N=None):
    """Checks an assignment of N rows (None: any), N x m or N (m = 1); returns N and m."""
    shape = idx.shape
    if len(shape) not in (1, 2):
        raise ValueError("idx must be N or N x m")
    if N is not None and shape[0] != N:
        raise ValueError(f"idx must have {N} rows, got {shape[0]}")
    _vector(idx, shape, torch.int32, "idx")
    if resp is not None:
        _vector(resp, shape, torch.float32, "resp")
    return shape if len(shape) == 2 else (shape[0], 1)


def _ld(t, name):
    """Elements from one row to the next of a matrix with a unit column stride."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with a unit column stride")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _dtype(t):
    dtype = _DTYPES.get(t.dtype)
    if dtype is None:
        raise TypeError(f"rows must be float32, bfloat16 or float16, got {t.dtype}")
    return dtype


def embed_problem(idx, K, scale, ldw, Y) -> gmm_embed_problem:
    """The problem of a gmm_embed or gmm_embed_backward call on these tensors."""
    N, D = Y.shape
    m = idx.shape[1] if idx.dim() == 2 else 1
    return gmm_embed_problem(N, m, K, D, _dtype(Y), scale, ldw, _ld(Y, "Y"))


def gmm_embed(W, idx, resp=None, scale=1.0, out=None, dev_flags=None, stream=None):
    """scale * sum_j resp_nj W[idx_nj]: the embedding of tokens (idx: N int32), or points put
    together from a codebook's or mixture's entries (idx, resp: N x m, as gmm_assign_topm and
    gmm_route return them; m <= 8).

    W: K x D float32, bfloat16 or float16, any row stride.  A choice of -1 is unused; resp None is
    weights of 1.  Returns N x D of W's type (into out when given).
    """
    if stream is not None:
        with _on(stream, W):
            return gmm_embed(W, idx, resp, scale, out, dev_flags)
    _same_device(W, idx, resp, out, dev_flags)
    N, m = _choices(idx, resp)
    ldw, ldy = _ld(W, "W"), None
    K, D = W.shape
    if dev_flags is not None:
        _vector(dev_flags, (1,), torch.int32, "dev_flags")
    dtype, device = _dtype(W), W.device
    if out is None:
        out, ldy = torch.empty(N, D, dtype=W.dtype, device=device), D
    elif out.dtype != W.dtype or out.shape != (N, D):
        raise ValueError("out must be N x D of W's type")
    p = _embed_of(N, m, K, D, dtype, _number(scale), ldw, _ld(out, "out") if ldy is None else ldy)
    _launch(load_library().gmm_embed, "gmm_embed", device, ctypes.byref(p), W.data_ptr(),
            idx.data_ptr(), _address(resp), out.data_ptr(), _address(dev_flags))
    return out


def gmm_embed_workspace_size(p: gmm_embed_problem) -> int:
    return _bytes(load_library().gmm_embed_workspace_size, "gmm_embed_workspace_size",
                  ctypes.byref(p))


def gmm_embed_backward(dY, idx, K, resp=None, W=None, scale=1.0, out=None, accumulate=False,
                       ws=None, dev_flags=None, stream=None, table=True):
    """(dW, dresp): the gradients of gmm_embed(W, idx, resp, scale) for its upstream gradient dY
    (N x D).

    dW: K x D of dY's type, or in out (of dY's type or float32); with accumulate it is added to
    what out holds, and rows that idx does not name are not touched.  dresp: of resp's shape, None
    unless W is given.  ws: a uint8 device tensor of gmm_embed_workspace_size bytes (allocated here
    when None).  table False: dresp alone, for a W that is not trained; dW is None and no workspace
    is used.
    """
    if stream is not None:
        with _on(stream, dY):
            return gmm_embed_backward(dY, idx, K, resp, W, scale, out, accumulate, ws, dev_flags,
                                      table=table)
    _same_device(dY, idx, resp, W, out, ws, dev_flags)
    ldy = _ld(dY, "dY")
    N, D = dY.shape
    m = _choices(idx, resp, N)[1]
    if dev_flags is not None:
        _vector(dev_flags, (1,), torch.int32, "dev_flags")
    K, dtype, device = int(K), _dtype(dY), dY.device
    ldw = D
    if W is not None:
        if W.dtype != dY.dtype or W.shape != (K, D):
            raise ValueError("W must be K x D of dY's type")
        ldw = _ld(W, "W")
    ldd = D
    if not table:
        if W is None or out is not None or accumulate:
            raise ValueError("without the table's gradient: W, and neither out nor accumulate")
        ws = None
    elif out is None:
        if accumulate:
            raise ValueError("accumulate adds to out, which is missing")
        out = torch.empty(K, D, dtype=dY.dtype, device=device)
    else:
        if out.dtype not in (dY.dtype, torch.float32) or out.shape != (K, D):
            raise ValueError("out must be K x D of dY's type or float32")
        ldd = _ld(out, "out")
    dresp = None if W is None else torch.empty(idx.shape, dtype=torch.float32, device=device)
    p = _embed_of(N, m, K, D, dtype, _number(scale), ldw, ldy)
    if table and ws is None:
        ws = torch.empty(_embed_bytes(N, m, K, D, dtype), dtype=torch.uint8, device=device)
    _launch(load_library().gmm_embed_backward, "gmm_embed_backward", device, ctypes.byref(p),
            dY.data_ptr(), idx.data_ptr(), _address(resp), _address(W), _address(out),
            _DTYPES[out.dtype] if table else dtype, ldd, int(bool(accumulate)), _address(dresp),
            _address(dev_flags), _address(ws), ws.numel() if table else 0)
    return out, dresp


class BeamStep(NamedTuple):
    """Results of gmm_beam_select for B groups, m candidates each."""

    scores: torch.Tensor  # B x m
    parent: torch.Tensor  # B x m int32: the candidate's beam, in its group
    token: torch.Tensor   # B x m int32


def gmm_beam_workspace_size(Z, w, m) -> int:
    """Bytes of gmm_beam_select's workspace for logits like Z, w beams and m candidates."""
    return _beam_bytes(Z.shape[0], w, m)


def gmm_beam_select(Z, scores, m=None, ended=None, end_id=0, scale=1.0, ws=None, dev_flags=None,
                    stream=None) -> BeamStep:
    """The m best continuations of each group of beams (m None: as many as beams), by
    scores[b, i] + log p of row b * w + i.

    Z: (B * w) x K logits, float32, bfloat16 or float16, any row stride; the logits are scale * Z.
    scores: B x w float32, -inf for no beam.  ended: B x w bool or uint8; a beam that has ended has
    the one candidate (itself, end_id) with its score as it is.  Candidates that run out have -inf,
    -1, -1.  w and m <= 32.  ws: a uint8 device tensor of gmm_beam_workspace_size bytes (allocated
    here when None).
    """
    if stream is not None:
        with _on(stream, Z):
            return gmm_beam_select(Z, scores, m, ended, end_id, scale, ws, dev_flags)
    r = _rows(Z, scale)
    _same_device(Z, scores, ended, ws, dev_flags)
    if scores.dim() != 2 or scores.numel() != Z.shape[0]:
        raise ValueError("scores must be B x w for B * w rows of logits")
    B, w = scores.shape
    _vector(scores, (B, w), torch.float32, "scores")
    if ended is not None:
        _vector(ended, (B, w), torch.bool if ended.dtype == torch.bool else torch.uint8, "ended")
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    m = w if m is None else int(m)
    device = Z.device
    if ws is None:
        ws = torch.empty(_beam_bytes(Z.shape[0], w, m), dtype=torch.uint8, device=device)
    out = torch.empty(B, m, dtype=torch.float32, device=device)
    parent = torch.empty(B, m, dtype=torch.int32, device=device)
    token = torch.empty(B, m, dtype=torch.int32, device=device)
    _launch(load_library().gmm_beam_select, "gmm_beam_select", Z.device, ctypes.byref(r),
            Z.data_ptr(), w, scores.data_ptr(), _address(ended), int(end_id), m, out.data_ptr(),
            parent.data_ptr(), token.data_ptr(), _address(dev_flags), ws.data_ptr(), ws.numel())
    return BeamStep(out, parent, token)


_STATE = struct.Struct("=6qi4x")  # gmm_beam_state


@functools.lru_cache(maxsize=4096)
def _state_layout(shape, stride, size, rows, dim):
    """A tensor's rows as gmm_beam_state, without the address; dim: that of its positions."""
    if len(shape) < 1 or shape[0] != rows:
        raise ValueError(f"a state must have {rows} rows, got {shape}")
    if dim is not None and not 0 < dim < len(shape):
        raise ValueError("dim must be a dimension of the state behind its rows")
    inner = 1 if dim is None else dim
    dense = 1  # elements of the dimensions behind, which must lie densely
    for d in range(len(shape) - 1, inner - 1, -1):
        if shape[d] > 1 and stride[d] != dense:
            raise ValueError("a state must be dense from its positions on")
        dense *= shape[d]
    outer, outer_stride = 1, 0
    for d in range(inner - 1, 0, -1):
        if shape[d] == 1:
            continue
        if outer > 1 and stride[d] != outer * outer_stride:
            raise ValueError("the dimensions before a state's positions must lie evenly")
        outer_stride = stride[d] if outer == 1 else outer_stride
        outer *= shape[d]
    count = 1 if dim is None else shape[dim]
    per = dense // count if count else 0
    return stride[0] * size, outer, outer_stride * size, count, per * size, int(dim is not None)


def gmm_beam_reorder(states, parent, lens=None, dim=None, dev_flags=None, stream=None):
    """The beams' states after their parents, in place: state[b, i] <- state[b, parent[b, i]].

    states: a tensor or a list of tensors of B * w rows each (a cache (B * w, heads, positions,
    width), token ids (B * w, positions), any type); parent: B x w int32, a beam of the same group,
    -1 to leave one as it is.  dim: the dimension of the positions, for all states or a list with
    one for each, None for states without; lens (B int32): how many positions of a group are used,
    those behind are left as they are.  w <= 32.  States must not overlap: one that serves twice is
    named once.
    """
    states = [states] if isinstance(states, torch.Tensor) else list(states)
    if stream is not None:
        with _on(stream, parent):
            return gmm_beam_reorder(states, parent, lens, dim, dev_flags)
    _same_device(parent, lens, dev_flags, *states)
    if parent.dim() != 2:
        raise ValueError("parent must be B x w")
    B, w = parent.shape
    _vector(parent, (B, w), torch.int32, "parent")
    _vector(lens, (B,), torch.int32, "lens")
    _vector(dev_flags, (1,), torch.int32, "dev_flags")
    dims = list(dim) if isinstance(dim, (list, tuple)) else [dim] * len(states)
    if len(dims) != len(states):
        raise ValueError("dim must be one for each state")
    packed, like, layout = [], None, None
    for t, d in zip(states, dims):  # (caches mostly have one shape)
        shape, stride = t.shape, t.stride()
        if like is None or shape != like[0] or stride != like[1] or (t.dtype, d) != like[2:]:
            like = shape, stride, t.dtype, d
            layout = _state_layout(shape, stride, t.element_size(), B * w, d)
        packed.append(_STATE.pack(t.data_ptr(), *layout))
    packed = b"".join(packed)
    _launch(load_library().gmm_beam_reorder, "gmm_beam_reorder", parent.device, B, w,
            parent.data_ptr(), _address(lens), len(states), packed, _address(dev_flags))


def gmm_device_status(ws, clear=True, stream=None):
    """(status, flags): waits for the stream and reads the workspace's device status word."""
    f = ctypes.c_uint32(0)
    rc = load_library().gmm_device_status(_ptr(ws), ws.numel(), _stream(stream), ctypes.byref(f),
                                          int(bool(clear)))
    return rc, int(f.value)


def gmm_trace_fused(start=None, stop=None):
    """Record torch.cuda.Event start/stop around every later fused-kernel launch (None: off)."""
    if start is None:
        _check(load_library().gmm_trace_fused(None, None), "gmm_trace_fused")
        return
    for e in (start, stop):
        if not e.cuda_event:
            e.record()  # torch creates the CUDA event lazily, on its first record
    _check(load_library().gmm_trace_fused(ctypes.c_void_p(start.cuda_event),
                                          ctypes.c_void_p(stop.cuda_event)), "gmm_trace_fused")


def gmm_set_wait_budget(ns=0):
    """Budget of every device-side wait in nanoseconds (0: the default, one second)."""
    _check(load_library().gmm_set_wait_budget(int(ns)), "gmm_set_wait_budget")


def gmm_launch_count() -> int:
    """Kernels the library has enqueued in this process so far."""
    c = ctypes.c_uint64(0)
    _check(load_library().gmm_launch_count(ctypes.byref(c)), "gmm_launch_count")
    return int(c.value)
