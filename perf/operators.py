"""Cases of the row-posterior operators and of the mixture-of-experts layer, with their plain forms.

Four operators over rows of logits (one logit per class: a mixture component, a vocabulary
entry, an expert):

  logprobs   log probability of a given class per row, the row's log-sum-exp and entropy,
             and its m most probable classes
  gradient   the gradient of all of those with respect to the logits
  route      the m most probable experts of a token and their weights
  experts    route, then the gated two-layer experts it chose, for a few tokens

With own = False a case runs in elementary torch operations in 32 bits, rounded once at the
end; with own = True it runs through soft_clustering_em_b200.gmm.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence being decoded: the sampled token's log probability and 8 alternatives
        dict(name="next_token_one", op="logprobs", N=1, K=131072, dtype="bf16", pad=0, m=8,
             scale=1.0, masks=False),
        # a decode batch that returns the 20 alternatives an API offers, at a temperature
        dict(name="next_token_batch", op="logprobs", N=64, K=131072, dtype="bf16", pad=0, m=20,
             scale=1.25, masks=False),
        # log probabilities of whole prompts or rollouts under a policy: no alternatives
        dict(name="prompt_scoring", op="logprobs", N=4096, K=131072, dtype="bf16", pad=0, m=0,
             scale=1.0, masks=False),
        # an odd vocabulary in padded rows, classes masked out by -inf and by the type's lowest
        # value, some rows with nothing left
        dict(name="ragged_masked", op="logprobs", N=1023, K=100003, dtype="f32", pad=5, m=5,
             scale=0.75, masks=True),
        # posteriors of a clustered data set (1e6 rows, 256 components) from given log-joints
        dict(name="posterior_rows", op="logprobs", N=1_000_000, K=256, dtype="f32", pad=0, m=2,
             scale=1.0, masks=False),
        # a training step: gradient of log probability, entropy and log-sum-exp penalties
        dict(name="train_gradient", op="gradient", N=4096, K=131072, dtype="bf16", pad=0, m=0,
             scale=1.0, masks=False),
        # distillation on the best few classes of 1,024-way rows, odd row count, masks
        dict(name="posterior_gradient", op="gradient", N=60_001, K=1024, dtype="f32", pad=0, m=4,
             scale=0.75, masks=True),
        # the router of one decode step
        dict(name="route_decode", op="route", N=8, K=64, dtype="bf16", m=8, renorm=True),
        # the router of a long prompt
        dict(name="route_prompt", op="route", N=16384, K=256, dtype="f32", m=8, renorm=False),
        # the whole layer for one token: latency
        dict(name="experts_one_token", op="experts", T=1, E=64, D=2048, F=1024, m=8,
             dtype="bf16", padded=0, renorm=True),
        # the whole layer for a decode batch: nearly every expert's weights are read
        dict(name="experts_batch", op="experts", T=32, E=128, D=2048, F=768, m=8, dtype="bf16",
             padded=0, renorm=True),
        # fewer, wider experts, an inner size that no tile divides, a padded batch
        dict(name="experts_padded", op="experts", T=100, E=32, D=4096, F=1432, m=4, dtype="f16",
             padded=7, renorm=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "gradient", "route", "experts", "experts"])
    if op == "experts":
        while True:
            T = _log_int(rng, 1, 128)
            E = _log_int(rng, 4, 128)
            D = 8 * _log_int(rng, 32, 512)
            F = 8 * _log_int(rng, 16, 256)
            if 2 * 3 * E * D * F <= 1_100_000_000:
                return dict(op=op, T=T, E=E, D=D, F=F, m=rng.randint(1, min(8, E)),
                            dtype=rng.choice(["bf16", "f16"]), padded=rng.randint(0, T // 4),
                            renorm=rng.random() < 0.5)
    if op == "route":
        return dict(op=op, N=_log_int(rng, 1, 16384), K=_log_int(rng, 8, 256),
                    dtype=rng.choice(["f32", "bf16", "f16"]), m=rng.randint(1, 8),
                    renorm=rng.random() < 0.5)
    K = _log_int(rng, 32, 262_144)
    N = _log_int(rng, 1, min(1_000_000, 256_000_000 // K))
    return dict(op=op, N=N, K=K, dtype=rng.choice(["f32", "bf16", "f16"]),
                pad=rng.choice([0, 0, 3, 8]), m=rng.choice([0, 1, 5, 8, 20]),
                scale=rng.choice([1.0, 0.75, 1.25]), masks=rng.random() < 0.4)


# ------------------------------------------------------------------ their inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed % (1 << 31))


def _logits(case, g):
    """N x K logits inside rows of K + pad, spread like a trained head's: a broad bulk and a few
    classes well above it."""
    N, K, t = case["N"], case["K"], _TYPES[case["dtype"]]
    Z = torch.randn(N, K + case.get("pad", 0), generator=g, device="cuda").mul_(2.5)
    rows = torch.arange(N, device="cuda")
    for lift in (9.0, 7.0, 4.0):
        Z[rows, torch.randint(K, (N,), generator=g, device="cuda")] += lift
    if case.get("masks"):
        cut = torch.rand(N, 1, generator=g, device="cuda")
        for r0 in range(0, N, 4096):
            part = Z[r0:r0 + 4096]
            drop = torch.rand(part.shape, generator=g, device="cuda") < 0.5 * cut[r0:r0 + 4096]
            low = torch.finfo(t).min if r0 % 8192 else -math.inf
            part.masked_fill_(drop, low)
        Z[5::97] = -math.inf  # rows that a mask leaves empty
    return Z.to(t)[:, :K]


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] in ("logprobs", "gradient"):
        N, K = case["N"], case["K"]
        s["Z"] = _logits(case, g)
        ids = torch.randint(K, (N,), generator=g, device="cuda", dtype=torch.int32)
        if case["masks"]:  # a label is a class that the mask leaves
            z = s["Z"].gather(1, ids.long()[:, None])[:, 0]
            ids = torch.where(z < -1e4, s["Z"].argmax(1).int(), ids)
        ids[3::11] = -1  # positions without a label (padding, prompts)
        s["ids"] = ids
        if case["op"] == "gradient":
            s["lse"], s["entropy"], s["top_idx"] = _saved(s["Z"], case["scale"], case["m"])
            for name in ("dlogp", "dentropy", "dlse"):
                s[name] = torch.randn(N, generator=g, device="cuda")
            s["dentropy"] *= 0.01
            s["dlse"] *= 0.01
            s["dtop"] = torch.randn(N, case["m"], generator=g, device="cuda") if case["m"] else None
        return s
    if case["op"] == "route":
        s["Z"] = (torch.randn(case["N"], case["K"], generator=g, device="cuda") * 1.5).to(
            _TYPES[case["dtype"]])
        return s
    T, E, D, F, t = case["T"], case["E"], case["D"], case["F"], _TYPES[case["dtype"]]
    s["Z"] = torch.randn(T, E, generator=g, device="cuda") * 1.5
    s["Z"][T - case["padded"]:] = -math.inf  # rows behind the last token go to no expert
    s["X"] = torch.randn(T, D, generator=g, device="cuda").to(t)
    s["W_up"] = torch.empty(E, 2 * F, D, dtype=t, device="cuda")
    s["W_down"] = torch.empty(E, D, F, dtype=t, device="cuda")
    for W, n in ((s["W_up"], D), (s["W_down"], F)):
        W.normal_(0, n ** -0.5, generator=g)
    return s


def _saved(Z, scale, m):
    """What the forward call of a training step leaves behind: lse, entropy, best classes."""
    lse, H, idx = [], [], []
    for r0 in range(0, Z.shape[0], 1024):
        z = Z[r0:r0 + 1024].double() * scale
        l = torch.logsumexp(z, 1)
        p = (z - l[:, None]).exp().nan_to_num(0.0)
        lse.append(l.float())
        H.append((l - (p * z.nan_to_num(0.0, neginf=0.0)).sum(1)).nan_to_num(0.0, neginf=0.0).float())
        if m:
            v, i = z.topk(min(m, z.shape[1]), 1)
            idx.append(i.int().masked_fill(v == -math.inf, -1))
    top = torch.cat(idx) if m else None
    return torch.cat(lse), torch.cat(H), top


# ------------------------------------------------------------------ one pass
def run(state):
    return {"logprobs": _run_logprobs, "gradient": _run_gradient, "route": _run_route,
            "experts": _run_experts}[state["op"]](state)


def _run_logprobs(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        r = G.gmm_logprobs(s["Z"], s["ids"], m=s["m"], scale=s["scale"])
        out = dict(logp=r.logp, entropy=r.entropy, lse=r.lse)
        return dict(out, top_idx=r.top_idx, top_logp=r.top_logp) if s["m"] else out
    z = s["Z"].float() * s["scale"]
    ids = s["ids"].long()
    top = z.amax(1)
    base = top.masked_fill(top == -math.inf, 0.0)
    d = z - base[:, None]
    e = d.exp()
    total = e.sum(1)
    lse = base + total.log()
    # sum of p * d over the classes that have a probability (0 * -inf is none)
    mean = (e * d.masked_fill(e == 0, 0.0)).sum(1) / total
    entropy = (total.log() - mean).masked_fill(top == -math.inf, 0.0)
    zi = d.gather(1, ids.clamp(min=0)[:, None])[:, 0]
    logp = (zi - total.log()).masked_fill(top == -math.inf, -math.inf).masked_fill(ids < 0, 0.0)
    out = dict(logp=logp, entropy=entropy, lse=lse)
    if s["m"]:
        v, i = _largest(z, s["m"])
        gone = v == -math.inf
        lp = (v - base[:, None] - total.log()[:, None]).masked_fill(gone, -math.inf)
        out.update(top_idx=i.int().masked_fill(gone, -1), top_logp=lp)
    return out


def _largest(z, m):
    """The m largest of each row, equal values in index order; past the row's end -1, -inf."""
    b = (z + 0.0).view(torch.int32)
    order = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
    key = (order << 32) | (0x7FFFFFFF - torch.arange(z.shape[1], device=z.device))
    i = 0x7FFFFFFF - (key.topk(min(m, z.shape[1]), 1).values & 0xFFFFFFFF)
    v = z.gather(1, i)
    short = m - i.shape[1]
    if short > 0:
        i = torch.nn.functional.pad(i, (0, short), value=-1)
        v = torch.nn.functional.pad(v, (0, short), value=-math.inf)
    return v, i


def _run_gradient(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        return G.gmm_logprobs_backward(
            s["Z"], s["ids"], s["lse"], dlogp=s["dlogp"], entropy=s["entropy"],
            dentropy=s["dentropy"], dlse=s["dlse"], top_idx=s["top_idx"], dtop=s["dtop"],
            scale=s["scale"])
    z = s["Z"].float() * s["scale"]
    ids = s["ids"].long()
    empty = s["lse"] == -math.inf
    logp = z - s["lse"].masked_fill(empty, 0.0)[:, None]
    p = logp.exp()
    a = s["dlogp"].masked_fill((ids < 0) | empty, 0.0)
    slope = s["dlse"] - a
    t = None
    if s["dtop"] is not None:
        t = s["dtop"].masked_fill(s["top_idx"] < 0, 0.0)
        slope = slope - t.sum(1)
    logp = logp.masked_fill_(p == 0, 0.0)
    grad = p * (slope[:, None] - s["dentropy"][:, None] * (logp + s["entropy"][:, None]))
    grad.scatter_add_(1, ids.clamp(min=0)[:, None], a[:, None])
    if t is not None:
        grad.scatter_add_(1, s["top_idx"].long().clamp(min=0), t)
    return (grad * s["scale"]).to(s["Z"].dtype)


def _route(Z, m, renorm):
    v, i = _largest(Z.float(), m)
    gone = v == -math.inf
    base = v[:, :1].masked_fill(gone[:, :1], 0.0)
    e = (v - base).exp()
    total = e.sum(1, keepdim=True) if renorm else (Z.float() - base).exp().sum(1, keepdim=True)
    return i.int().masked_fill(gone, -1), (e / total).masked_fill(gone, 0.0)


def _run_route(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        idx, resp = G.gmm_route(s["Z"], s["m"], renorm=s["renorm"])
    else:
        idx, resp = _route(s["Z"], s["m"], s["renorm"])
    return dict(idx=idx, resp=resp)


def _run_experts(s):
    X, W_up, W_down = s["X"], s["W_up"], s["W_down"]
    if own:
        from soft_clustering_em_b200 import gmm as G

        idx, resp = G.gmm_route(s["Z"], s["m"], renorm=s["renorm"])
        return dict(idx=idx, resp=resp, y=G.gmm_moe(X, idx, resp, W_up, W_down))
    idx, resp = _route(s["Z"], s["m"], s["renorm"])
    (T, D), (E, _, F), m = X.shape, W_down.shape, s["m"]
    e, x = idx.long().clamp(min=0), X.float()
    if T * m < E:  # the chosen experts' weights, one copy for each of a token's choices
        up = (W_up[e.flatten()].float() @ x.repeat_interleave(m, 0)[:, :, None])[:, :, 0]
        h = torch.nn.functional.silu(up[:, :F]) * up[:, F:] * resp.flatten()[:, None]
        y = (W_down[e.flatten()].float() @ h[:, :, None]).view(T, m, D).sum(1)
    else:  # every expert on every token, weighted by what the router gave it (mostly 0)
        up = (x @ W_up.float().view(E * 2 * F, D).T).view(T, E, 2 * F)
        weight = torch.zeros(T, E, device=X.device).scatter_add_(1, e, resp)
        h = torch.nn.functional.silu(up[:, :, :F]) * up[:, :, F:] * weight[:, :, None]
        y = torch.matmul(h.transpose(0, 1), W_down.float().transpose(1, 2)).sum(0)
    return dict(idx=idx, resp=resp, y=y.to(X.dtype))


# ------------------------------------------------------------------ the work of a pass
def work(case):
    m = case["m"]
    if case["op"] == "experts":
        T, E, D, F = case["T"] - case["padded"], case["E"], case["D"], case["F"]
        active = E * (1.0 - (1.0 - m / E) ** T)  # experts that a token chooses, on average
        return dict(bytes=2 * 3 * D * F * active + 2 * 2 * case["T"] * D + 4 * case["T"] * E
                    + 8 * case["T"] * m, flops=2.0 * 3 * D * F * T * m)
    N, K, b = case["N"], case["K"], _BYTES[case["dtype"]]
    if case["op"] == "gradient":
        return dict(bytes=2.0 * N * K * b + N * (24 + 8 * m), flops=7.0 * N * K)
    out = 8 * m + (0 if case["op"] == "route" else 16)
    return dict(bytes=1.0 * N * K * b + N * out, flops=5.0 * N * K)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "experts":
        return _exact_experts(s)
    if case["op"] == "route":
        return dict(idx=None, resp=_exact_weights(s["Z"], case["m"], case["renorm"])[1])
    parts = []
    for r0 in range(0, case["N"], 2048 if case["K"] > 2048 else 65536):
        rows = slice(r0, r0 + (2048 if case["K"] > 2048 else 65536))
        parts.append((_exact_logprobs if case["op"] == "logprobs" else _exact_gradient)(s, rows))
    if case["op"] == "gradient":
        return torch.cat(parts)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return dict(out, top_idx=None) if case["m"] else out


def _exact_logprobs(s, rows):
    z = s["Z"][rows].double() * s["scale"]
    ids = s["ids"][rows].long()
    q = torch.log_softmax(z, 1)  # NaN in rows with nothing left
    empty = z.max(1).values == -math.inf
    logp = torch.where(ids < 0, 0.0, q.gather(1, ids.clamp(min=0).view(-1, 1)).view(-1))
    logp = torch.where(empty & (ids >= 0), -math.inf, logp)
    H = -torch.special.xlogy(q.exp(), q.exp()).sum(1)
    out = dict(logp=logp, entropy=torch.where(empty, 0.0, H), lse=torch.logsumexp(z, 1))
    if s["m"]:
        k = min(s["m"], z.shape[1])
        best = torch.where(empty[:, None], -math.inf, q.topk(k, 1).values)
        out["top_logp"] = torch.cat([best, best.new_full((len(best), s["m"] - k), -math.inf)], 1)
    return out


def _exact_gradient(s, rows):
    z = s["Z"][rows].double() * s["scale"]
    q = torch.log_softmax(z, 1)
    p = q.exp().nan_to_num(0.0)
    n = torch.arange(len(z), device=z.device)
    H = s["entropy"][rows].double()[:, None]
    dH, dl = (s[k][rows].double()[:, None] for k in ("dentropy", "dlse"))
    out = dl * p - dH * (torch.special.xlogy(p, p) + p * H)
    live = (s["lse"][rows] != -math.inf).double()
    for ids, w in [(s["ids"], s["dlogp"])] + (
            [(s["top_idx"][:, j], s["dtop"][:, j]) for j in range(s["m"])] if s["m"] else []):
        i, a = ids[rows].long(), w[rows].double() * live
        a = torch.where(i < 0, 0.0, a)
        out -= a[:, None] * p
        out[n, i.clamp(min=0)] += a
    return out * s["scale"]


def _exact_weights(Z, m, renorm):
    z = Z.double()
    v, i = torch.sort(z, dim=1, descending=True, stable=True)
    v, i = v[:, :m], i[:, :m]
    total = torch.logsumexp(v if renorm else z, 1, keepdim=True)
    return i, torch.where(v == -math.inf, 0.0, (v - total).exp()).nan_to_num(0.0)


def _exact_experts(s):
    idx, w = _exact_weights(s["Z"], s["m"], s["renorm"])
    x = s["X"].double()
    F = s["F"]
    y = torch.zeros_like(x)
    for e in range(s["E"]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            up = x[t] @ s["W_up"][e].double().T
            h = up[:, :F] * torch.sigmoid(up[:, :F]) * up[:, F:]
            y.index_add_(0, t, w[t, j][:, None] * (h @ s["W_down"][e].double().T))
    return dict(idx=None, resp=w, y=y)
