"""Row log probabilities, their gradient, routing and few-token experts, in float64 numpy.

The logits z = float32(scale) * float32(x) are rounded to float32 as the library defines them
(the order of the alternatives is the order of those values); everything after that is float64.
"""
import numpy as np


def logits(x, scale=1.0):
    """z of a row set: float32 values, as float64."""
    with np.errstate(over="ignore"):
        return (np.asarray(x, np.float32) * np.float32(scale)).astype(np.float64)


def _rowwise(z):
    bad = np.isnan(z).any(1) | (z == np.inf).any(1)
    M = np.where(bad, 0.0, z.max(1))
    empty = M == -np.inf
    base = np.where(empty, 0.0, M)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        lse = base + np.log(np.exp(z - base[:, None]).sum(1))
    return bad, empty, np.where(bad, np.nan, lse)


def order(z, m):
    """Indices of the m largest of each row, equal values in index order, -1 past the last
    class that is not masked."""
    idx = np.full((z.shape[0], m), -1, np.int32)
    for n, row in enumerate(z):
        best = np.lexsort((np.arange(len(row)), -row))[:m]
        best = best[row[best] > -np.inf]
        idx[n, :len(best)] = best
    return idx


def logprobs(x, ids, m, scale=1.0):
    """(logp, entropy, lse, top_idx, top_logp)."""
    z = logits(x, scale)
    bad, empty, lse = _rowwise(z)
    rows = np.arange(len(z))
    with np.errstate(invalid="ignore"):
        lp = np.where((z == -np.inf) | empty[:, None], -np.inf, z - lse[:, None])
        p = np.exp(lp)
        H = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(1)
    H = np.where(bad, np.nan, H)
    logp = np.zeros(len(z))
    if ids is not None:
        ids = np.asarray(ids)
        legal = (ids >= 0) & (ids < z.shape[1])
        logp = np.where(legal, lp[rows, np.where(legal, ids, 0)], np.nan)
        logp = np.where(bad, np.nan, logp)
        logp = np.where(ids == -1, 0.0, logp)
    idx = order(np.where(np.isnan(z), -np.inf, z), m)
    idx[bad] = -1
    top = np.where(idx >= 0, np.take_along_axis(lp, np.maximum(idx, 0), 1), -np.inf)
    top[bad] = np.nan
    return logp, H, lse, idx, top


def gradient(x, ids, lse, entropy, dlogp, dentropy, dlse, top_idx, dtop, scale=1.0):
    """Gradient with respect to x; lse and entropy are taken as given."""
    z = logits(x, scale)
    N, K = z.shape
    lse = np.asarray(lse, np.float64)
    empty = lse == -np.inf
    zero = np.zeros(N)
    with np.errstate(invalid="ignore", over="ignore"):
        lp = np.where(empty[:, None], -np.inf, z - lse[:, None])
        p = np.exp(lp)
    slope = zero + (0 if dlse is None else dlse)
    direct = np.zeros((N, K))

    def named(idx, g):
        nonlocal slope
        idx = np.asarray(idx)
        use = (idx >= 0) & (idx < K) & ~empty
        g = np.where(use, g, 0.0)
        np.add.at(direct, (np.arange(N), np.where(use, idx, 0)), g)
        slope = slope - g

    if dlogp is not None:
        named(ids, dlogp)
    if dtop is not None:
        for j in range(dtop.shape[1]):
            named(top_idx[:, j], dtop[:, j])
    h = zero if dentropy is None else np.asarray(dentropy, np.float64)
    H = zero if entropy is None else np.asarray(entropy, np.float64)
    with np.errstate(invalid="ignore"):
        inner = np.where(p > 0, slope[:, None] - h[:, None] * (np.where(p > 0, lp, 0.0)
                                                               + H[:, None]), 0.0)
        g = np.where(p > 0, p * inner, 0.0) + direct
    g[np.isnan(lse)] = np.nan
    return np.float64(np.float32(scale)) * g


def route(x, m, renorm, scale=1.0):
    """(idx, resp)."""
    z = logits(x, scale)
    bad, empty, lse = _rowwise(z)
    idx = order(np.where(np.isnan(z), -np.inf, z), m)
    idx[bad] = -1
    zj = np.where(idx >= 0, np.take_along_axis(z, np.maximum(idx, 0), 1), -np.inf)
    if renorm:
        lse = _rowwise(zj)[2]
    with np.errstate(invalid="ignore"):
        resp = np.where(idx >= 0, np.exp(zj - np.where(np.isinf(lse), 0.0, lse)[:, None]), 0.0)
    resp[bad] = np.nan
    return idx, resp


def activation(x, act):
    with np.errstate(over="ignore"):
        if act == 0:
            return x / (1.0 + np.exp(-x))
        return 0.5 * x * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)))


def moe(X, idx, resp, W_up, W_down, act=0):
    """(Y, bound): Y and, for each element, the sum of the magnitudes that its products add up
    to (the scale of a float32 summation error)."""
    X = np.asarray(X, np.float64)
    E, D, F = W_down.shape
    Y, bound = np.zeros((len(X), D)), np.zeros((len(X), D))
    for t in range(len(X)):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            up, size = W_up[e] @ X[t], np.abs(W_up[e]) @ np.abs(X[t])
            a = activation(up[:F], act)
            Y[t] += resp[t, j] * (W_down[e] @ (a * up[F:]))
            h = np.abs(a) * size[F:] + 1.13 * size[:F] * np.abs(up[F:])
            bound[t] += abs(resp[t, j]) * (np.abs(W_down[e]) @ h)
    return Y, bound


def to_type(v, dtype):
    """v (float64) rounded once to bf16 or f16, as float64."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(v, np.float64))
    return t.to({"bf16": torch.bfloat16, "f16": torch.float16}[dtype]).double().numpy()


def moe_limit(X, idx, resp, W_up, W_down, act, dtype):
    """(Y, limit): Y, and for each token the largest 2-norm that Y's error may have.

    A product of the tensor cores over n elements is off by at most (n / 16 + 32) 2^-23 of its
    magnitudes (16 elements at a time, a step rounded or cut at 2^-23), an activation by 2^-21 in
    relation, the inner activation h kept in two halves by 2^-17 (bf16) or 2^-22 and 2^-36 (f16).
    An error d of h reaches y as W_down d, whose norm is at most the spectral norm times d's.
    With e for all of this in y, the rounded y is off by at most |round(y) - y| + 2 |e|: the
    distance to the nearest value of the type changes by |e| at most.
    """
    X, resp = np.asarray(X, np.float64), np.asarray(resp, np.float64)
    E, D, F = W_down.shape
    rel, low = (2.0 ** -17, 0.0) if dtype == "bf16" else (2.0 ** -22, 2.0 ** -36)
    up_c, down_c = (D / 16 + 32) * 2.0 ** -23, (F / 16 + 32) * 2.0 ** -23
    Y, _ = moe(X, idx, resp, W_up, W_down, act)
    limit = np.linalg.norm(to_type(Y, dtype) - Y, axis=1)
    for t in range(len(X)):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            up, off = W_up[e] @ X[t], up_c * (np.abs(W_up[e]) @ np.abs(X[t]))
            a = activation(up[:F], act)
            h = a * up[F:]
            dh = (1.13 * off[:F] + 2.0 ** -21 * np.abs(a)) * np.abs(up[F:]) + np.abs(a) * off[F:]
            dh = dh + rel * np.abs(h) + low
            dy = np.linalg.norm(W_down[e], 2) * np.linalg.norm(dh)
            dy += down_c * np.linalg.norm(np.abs(W_down[e]) @ np.abs(h))
            limit[t] += 2 * abs(resp[t, j]) * dy
    return Y, limit
