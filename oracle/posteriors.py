"""Row log probabilities, their gradient, routing and few-token experts, in float64 numpy.

The logits z = float32(scale) * float32(x) are rounded to float32 as the library defines them
(the order of the alternatives is the order of those values); everything after that is float64.
"""
import numpy as np


def logits(x, scale=1.0):
    """z of a row set: float32 values, as float64."""
    with np.errstate(over="ignore"):
        return (np.asarray(x, np.float32) * np.float32(scale)).astype(np.float64)


def _sums(z):
    """(bad, empty, base, log sum of e^{z - base}) per row, base the largest z (or 0).  The two
    are kept apart: beside a base of -3e38 the logarithm would be lost."""
    bad = np.isnan(z).any(1) | (z == np.inf).any(1)
    M = np.where(bad, 0.0, z.max(1))
    empty = M == -np.inf
    base = np.where(empty, 0.0, M)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        log_sum = np.log(np.exp(z - base[:, None]).sum(1))
    return bad, empty, base, np.where(bad, np.nan, log_sum)


def _rowwise(z):
    bad, empty, base, log_sum = _sums(z)
    return bad, empty, base + log_sum


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
    bad, empty, base, log_sum = _sums(z)
    lse = base + log_sum
    rows = np.arange(len(z))
    with np.errstate(invalid="ignore"):
        lp = np.where((z == -np.inf) | empty[:, None], -np.inf,
                      (z - base[:, None]) - log_sum[:, None])
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
    return _gradient(logits(x, scale), ids, lse, entropy, dlogp, dentropy, dlse, top_idx, dtop,
                     scale)


def _gradient(z, ids, lse, entropy, dlogp, dentropy, dlse, top_idx, dtop, scale):
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


FAR_LSE = 1024.0  # rows with an |lse| from here on are summed once more by the gradient


def gradient_limit(x, ids, lse, entropy, dlogp, dentropy, dlse, top_idx, dtop, scale, eps,
                   smallest):
    """(gradient, tolerance per entry) for a gradient that is rounded to a type of this eps and
    smallest normal number.  u = 2^-24:
      log p  from the given lse: off by u (|z| + |lse| + |log p|).  In rows with |lse| >= FAR_LSE
             from the row's own sum: by u (4 |z - max| + K / 32 + 64), and lse is exact here;
             p in relation by that, 3 u |log p| and 2^-21 (the hardware exponential), and whole
             below 2^-126;
      sums   of the m + 4 terms in brackets: (8 + m) u of their magnitudes;
      named  entries alone (a label's, an alternative's): (m + 4) u of the magnitudes given to
             them;
    and half a step of the type.
    """
    u = 2.0 ** -24
    z = logits(x, scale)
    N, K = z.shape
    lse = np.asarray(lse, np.float64)
    far = np.isfinite(lse) & (np.abs(lse) >= FAR_LSE)
    _, _, base, log_sum = _sums(z)
    z = np.where(far[:, None], z - base[:, None], z)  # the same row, its largest z at 0
    lse = np.where(far, log_sum, lse)
    want = _gradient(z, ids, lse, entropy, dlogp, dentropy, dlse, top_idx, dtop, scale)
    live = np.isfinite(z) & np.isfinite(lse)[:, None]
    zz, ll = np.where(live, z, 0.0), np.where(np.isfinite(lse), lse, 0.0)[:, None]
    lp = np.where(live, zz - ll, -200.0)
    p = np.where(live, np.exp(np.minimum(lp, 0.0)), 0.0)
    zero = np.zeros(N)
    h = zero if dentropy is None else np.abs(np.asarray(dentropy, np.float64))
    H = zero if entropy is None else np.abs(np.nan_to_num(np.asarray(entropy, np.float64)))
    mag = zero + sum(np.abs(d) for d in (dlogp, dlse) if d is not None)
    m = 0 if dtop is None else dtop.shape[1]
    named = np.zeros((N, K))
    pairs = [] if dlogp is None else [(ids, dlogp)]
    pairs += [(top_idx[:, j], dtop[:, j]) for j in range(m)]
    for i, d in pairs:
        use = (i >= 0) & (i < K)
        np.add.at(named, (np.arange(N), np.where(use, i, 0)), np.where(use, np.abs(d), 0.0))
    if m:
        mag = mag + np.abs(dtop).sum(1)
    terms = mag[:, None] + h[:, None] * (np.abs(lp) + H[:, None])
    off_lp = np.where(far[:, None], u * (4 * np.abs(zz) + K / 32 + 64),
                      u * (np.abs(zz) + np.abs(ll) + np.abs(lp)))
    off_lp = np.where(live, off_lp, 0.0)
    rel_p = off_lp + 3 * u * np.abs(lp) + 2.0 ** -21
    tol = p * (terms * (rel_p + (8 + m) * u) + h[:, None] * off_lp) + live * terms * 2.0 ** -126
    tol = scale * (tol + (m + 4) * u * named)
    return want, tol * 1.01 + np.abs(want) * (eps / 2 + 2 * u) + smallest * eps


def route(x, m, renorm, scale=1.0):
    """(idx, resp)."""
    z = logits(x, scale)
    bad, empty, base, log_sum = _sums(z)
    idx = order(np.where(np.isnan(z), -np.inf, z), m)
    idx[bad] = -1
    zj = np.where(idx >= 0, np.take_along_axis(z, np.maximum(idx, 0), 1), -np.inf)
    if renorm:
        _, _, base, log_sum = _sums(zj)
    log_sum = np.where(np.isinf(log_sum), 0.0, log_sum)
    with np.errstate(invalid="ignore"):
        resp = np.where(idx >= 0, np.exp((zj - base[:, None]) - log_sum[:, None]), 0.0)
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
