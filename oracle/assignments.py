"""Lookups by assignment, router losses and beam search, in float64 numpy.

Arguments and results are laid out as the library's; a choice outside [0, K) is left out.
"""
import numpy as np


def _legal(idx, K):
    idx = np.asarray(idx).reshape(len(idx), -1)
    ok = (idx >= 0) & (idx < K)
    return np.where(ok, idx, 0), ok


def _weights(resp, ok):
    r = np.ones(ok.shape) if resp is None else np.asarray(resp, np.float64).reshape(ok.shape)
    return np.where(ok, r, 0.0)


def embed(W, idx, resp=None, scale=1.0):
    """(Y, sum of the terms' magnitudes)."""
    W = np.asarray(W, np.float64)
    k, ok = _legal(idx, len(W))
    terms = W[k] * _weights(resp, ok)[:, :, None]
    terms = np.where(ok[:, :, None], terms, 0.0) * np.float64(np.float32(scale))
    return terms.sum(1), np.abs(terms).sum(1)


def embed_backward(dY, idx, K, resp=None, scale=1.0):
    """(dW, sum of the terms' magnitudes, how often each class is named)."""
    dY = np.asarray(dY, np.float64) * np.float64(np.float32(scale))
    k, ok = _legal(idx, K)
    r = _weights(resp, ok)
    dW, size = np.zeros((K, dY.shape[1])), np.zeros((K, dY.shape[1]))
    for j in range(k.shape[1]):
        n = ok[:, j]
        term = dY[n] * r[n, j, None]
        np.add.at(dW, k[n, j], term)
        np.add.at(size, k[n, j], np.abs(term))
    return dW, size, np.bincount(k[ok], minlength=K)


def embed_dresp(dY, W, idx, scale=1.0):
    """(dresp, sum of the terms' magnitudes), N x m."""
    dY, W = np.asarray(dY, np.float64), np.asarray(W, np.float64)
    k, ok = _legal(idx, len(W))
    terms = dY[:, None] * W[k] * np.float64(np.float32(scale))
    return np.where(ok, terms.sum(2), 0.0), np.where(ok, np.abs(terms).sum(2), 0.0)


def _softmax(x, scale):
    """(p, lse, empty, bad, log p) of the rows of float32 logits x.  (log p is not formed from lse:
    beside logits of -3e38 the logarithm of the sum would be lost.)"""
    z = np.asarray(x, np.float64) * np.float64(np.float32(scale))
    with np.errstate(over="ignore"):
        f = np.asarray(x, np.float32) * np.float32(scale)  # decides what is masked
    bad = np.isnan(f).any(1) | (f == np.inf).any(1)
    empty = ~bad & (f == -np.inf).all(1)
    top = np.where(bad | empty, 0.0, np.where(np.isnan(z), 0.0, z).max(1))
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        e = np.exp(z - top[:, None])
        S = e.sum(1)
        p = np.where(bad[:, None], np.nan, np.where(empty[:, None], 0.0, e / S[:, None]))
        lse = np.where(bad, np.nan, top + np.log(S))
        logp = np.where(bad[:, None], np.nan, (z - top[:, None]) - np.log(S)[:, None])
    return p, lse, empty, bad, logp


def _segments(N, offsets, mask, empty):
    """A list of the rows that count, per segment."""
    o = [0, N] if offsets is None else [int(v) for v in offsets]
    keep = ~empty if mask is None else ~empty & (np.asarray(mask) != 0)
    return [np.arange(lo, hi)[keep[lo:hi]] for lo, hi in zip(o[:-1], o[1:])]


def route_loss(x, idx, offsets=None, mask=None, scale=1.0):
    """(balance, z, load, counts, rows)."""
    p, lse, empty, _, _ = _softmax(x, scale)
    K, m = p.shape[1], np.asarray(idx).shape[1]
    balance, z, load, counts, rows = [], [], [], [], []
    for n in _segments(len(p), offsets, mask, empty):
        L = max(len(n), 1)
        k, ok = _legal(np.asarray(idx)[n], K) if len(n) else (np.zeros((0, m), int), None)
        c = np.bincount(k[ok], minlength=K) if len(n) else np.zeros(K, int)
        P = p[n].sum(0) / L
        load.append(P)
        counts.append(c)
        rows.append(len(n))
        balance.append(K * (c / (m * L) * P).sum())
        z.append((lse[n] ** 2).sum() / L)
    return tuple(np.array(v) for v in (balance, z, load, counts, rows))


def route_backward(x, idx, dresp=None, renorm=False, counts=None, rows=None, dbalance=None,
                   dz=None, offsets=None, mask=None, scale=1.0):
    """(dx, sum of the terms' magnitudes)."""
    p, lse, empty, bad, _ = _softmax(x, scale)
    N, K = p.shape
    m = np.asarray(idx).shape[1]
    grad, size = np.zeros((N, K)), np.zeros((N, K))
    involved = np.zeros(N, bool)
    if dbalance is not None or dz is not None:
        for s, n in enumerate(_segments(N, offsets, mask, empty)):
            L = max(int(rows[s]), 1)
            involved[n] = True
            if dbalance is not None:
                g = float(dbalance[s]) * K * np.asarray(counts[s], np.float64) / (m * float(L) ** 2)
                inner = p[n] @ g
                grad[n] += p[n] * (g - inner[:, None])
                size[n] += p[n] * (np.abs(g) + (p[n] @ np.abs(g))[:, None])
            if dz is not None:
                pull = 2.0 * float(dz[s]) / L * lse[n]
                grad[n] += p[n] * pull[:, None]
                size[n] += p[n] * np.abs(pull)[:, None]
    if dresp is not None:
        k, ok = _legal(idx, K)
        involved |= ok.any(1)
        d = np.where(ok, np.asarray(dresp, np.float64), 0.0)
        for n in np.nonzero(ok.any(1) & ~empty & ~bad)[0]:
            pk = np.where(ok[n], p[n, k[n]], 0.0)
            if renorm:
                q = np.where(ok[n], pk / pk.sum(), 0.0)
                a = q * (d[n] - (q * d[n]).sum())
                b = q * (np.abs(d[n]) + (q * np.abs(d[n])).sum())
            else:
                a, b = pk * d[n], np.abs(pk * d[n])
                grad[n] -= p[n] * a.sum()
                size[n] += p[n] * b.sum()
            np.add.at(grad[n], k[n][ok[n]], a[ok[n]])
            np.add.at(size[n], k[n][ok[n]], b[ok[n]])
    grad[bad & involved] = np.nan
    grad[(bad & ~involved) | empty] = 0.0
    c = np.float64(np.float32(scale))
    return grad * c, size * c


def beam_scores(x, scores, ended=None, end_id=0, scale=1.0):
    """B x w x K: every candidate's score, -inf where there is none."""
    B, w = np.asarray(scores).shape
    _, _, empty, _, logp = _softmax(x, scale)
    with np.errstate(over="ignore", invalid="ignore"):
        masked = np.asarray(x, np.float32) * np.float32(scale) == -np.inf
        q = np.where(masked | empty[:, None], -np.inf, logp)
    q = q.reshape(B, w, -1)
    s = np.asarray(scores, np.float64)[:, :, None]
    q = np.where(s == -np.inf, -np.inf, q + np.where(s == -np.inf, 0.0, s))
    if ended is not None:
        alone = np.full_like(q, -np.inf)
        alone[:, :, end_id] = s[:, :, 0]
        q = np.where(np.asarray(ended, bool)[:, :, None], alone, q)
    return q


def beam_select(x, scores, m, ended=None, end_id=0, scale=1.0):
    """(scores, parent, token): equal scores in the order of beam, then logit, then class."""
    q = beam_scores(x, scores, ended, end_id, scale)
    B, w, K = q.shape
    out = np.full((B, m), -np.inf), np.full((B, m), -1), np.full((B, m), -1)
    z = (np.asarray(x, np.float32) * np.float32(scale)).reshape(B, w * K)
    i = np.repeat(np.arange(w), K)
    for b in range(B):
        v = q[b].ravel()
        if np.isnan(v).any():
            out[0][b] = np.nan
            continue
        best = np.lexsort((np.arange(w * K), -z[b], i, -v))[:m]
        best = best[v[best] > -np.inf]
        for o, val in zip(out, (v[best], best // K, best % K)):
            o[b, :len(best)] = val
    return out


def beam_reorder(state, parent, lens=None, dim=None):
    """The state (rows b w + i first) after its beams' parents."""
    B, w = np.asarray(parent).shape
    out = state.copy()
    for b in range(B):
        for i, p in enumerate(parent[b]):
            if not 0 <= p < w:
                continue
            at = [b * w + i] + [slice(None)] * (state.ndim - 1)
            if lens is not None and dim is not None:
                at[dim] = slice(0, min(max(int(lens[b]), 0), state.shape[dim]))
            src = [b * w + p] + at[1:]
            out[tuple(at)] = state[tuple(src)]
    return out
