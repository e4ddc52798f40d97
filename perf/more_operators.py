"""Cases of the operators around a vocabulary and a router, with their plain forms.

  embed       rows of a table chosen by an assignment (token ids; a codebook's best entries with
              their weights), summed and scaled
  embed_grad  the gradient of that with respect to the table, and to the weights
  beam        the best continuations of each group of beams
  reorder     the beams' states (caches, token histories) after their parents
  balance     how a router loads its experts: counts, mean probabilities, balance and z losses
  route_grad  the gradient of those losses and of the routed weights with respect to the logits

With own = False a case runs in elementary torch operations in 32 bits (scores next to one
another in 64), rounded once at the end; with own = True through soft_clustering_em_b200.gmm.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the input of one decode step: 8 tokens, latency
        dict(name="embed_decode", op="embed", N=8, m=1, K=131072, D=2048, dtype="bf16", pad=0,
             weights=False),
        # points of a clustered data set put together again from their two best components
        dict(name="embed_mixture", op="embed", N=1_000_000, m=2, K=4096, D=96, dtype="f32", pad=0,
             weights=True),
        # a training step's tokens over a vocabulary: the whole table's gradient
        dict(name="embed_grad_tokens", op="embed_grad", N=16384, m=1, K=131072, D=2048,
             dtype="bf16", pad=0, weights=False, add=False),
        # a codebook learnt from soft assignments, added to what earlier batches gave; odd sizes
        dict(name="embed_grad_mixture", op="embed_grad", N=200_001, m=2, K=4096, D=96,
             dtype="f32", pad=0, weights=True, add=True),
        # one request with 4 beams that asks for twice as many candidates
        dict(name="beam_one", op="beam", B=1, w=4, K=131072, dtype="bf16", pad=0, m=8,
             scale=1.0, masks=False),
        # a batch with an odd vocabulary in padded rows, at a temperature, classes masked out,
        # beams that have ended and beams that are none yet
        dict(name="beam_batch", op="beam", B=64, w=8, K=100003, dtype="f32", pad=5, m=16,
             scale=0.75, masks=True),
        # caches of one request, a short prompt in a longer buffer
        dict(name="reorder_one", op="reorder", B=1, w=4, n=8, H=8, T=512, d=128, dtype="bf16",
             least=64, most=128),
        # caches of a batch, sequences of different lengths
        dict(name="reorder_batch", op="reorder", B=16, w=8, n=4, H=8, T=1024, d=128,
             dtype="bf16", least=300, most=1024),
        # a small router's batch, one loss over all of it
        dict(name="balance_small", op="balance", N=512, K=8, dtype="f32", m=2, S=0, masks=False),
        # packed sequences, a loss for each, some positions padding
        dict(name="balance_sequences", op="balance", N=65536, K=256, dtype="f32", m=8, S=16,
             masks=True),
        # the router's gradient in a small training step
        dict(name="route_grad_small", op="route_grad", N=2048, K=64, dtype="bf16", m=6, S=0,
             masks=False, renorm=True),
        # and for packed sequences over many experts
        dict(name="route_grad_sequences", op="route_grad", N=65536, K=256, dtype="f32", m=8, S=16,
             masks=True, renorm=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "beam", "reorder", "balance", "route_grad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("embed", "embed_grad"):
        K = _log_int(rng, 16, 262_144)
        D = _log_int(rng, 8, min(8192, 200_000_000 // K))
        if rng.random() < 0.7:  # widths are mostly whole vectors
            D = (D + 7) // 8 * 8
        m = rng.choice([1, 1, 2, 4])
        N = _log_int(rng, 1, min(500_000, 60_000_000 // (D * m)))
        case = dict(op=op, N=N, m=m, K=K, D=D, dtype=dtype, pad=rng.choice([0, 0, 8, 3]),
                    weights=m > 1 or rng.random() < 0.2)
        return dict(case, add=rng.random() < 0.4) if op == "embed_grad" else case
    if op == "beam":
        w, K = rng.randint(1, 16), _log_int(rng, 50, 262_144)
        B = _log_int(rng, 1, max(1, min(128, 50_000_000 // (w * K))))
        return dict(op=op, B=B, w=w, K=K, dtype=dtype, pad=rng.choice([0, 0, 3, 8]),
                    m=rng.randint(w, min(32, 2 * w)), scale=rng.choice([1.0, 0.75, 1.25]),
                    masks=rng.random() < 0.4)
    if op == "reorder":
        w, H, d = rng.randint(2, 16), rng.randint(1, 16), rng.choice([64, 80, 128, 576])
        n, B = rng.randint(1, 12), _log_int(rng, 1, 32)
        T = _log_int(rng, 16, max(16, min(16384, 250_000_000 // (n * B * w * H * d))))
        most = _log_int(rng, 1, T)
        return dict(op=op, B=B, w=w, n=n, H=H, T=T, d=d, dtype=dtype,
                    least=_log_int(rng, 1, most), most=most)
    N, K = _log_int(rng, 1, 65536), _log_int(rng, 4, 256)
    case = dict(op=op, N=N, K=K, dtype=dtype, m=rng.randint(1, min(8, K)),
                S=rng.choice([0, 0, 1, 5, 64]), masks=rng.random() < 0.5)
    return dict(case, renorm=rng.random() < 0.5) if op == "route_grad" else case


# ------------------------------------------------------------------ their inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed % (1 << 31))


def _randn(g, *shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _classes(N, m, K, g):
    """N x m different classes per row, the k-th most frequent about k times as rare as the
    first (as tokens are), spread over the table; every 41st row has none (padding)."""
    u = torch.rand(N, 1, generator=g, device="cuda")
    rank = (u * math.log(K + 1)).exp().long().clamp(1, K) - 1
    rank = (rank + torch.arange(m, device="cuda") * max(1, K // m)) % K
    step = next(p for p in range(40_503, 41_503) if math.gcd(p, K) == 1)
    idx = (rank * step % K).int()
    idx[40::41] = -1
    return idx


def _rows_of(t, pad):
    """The same values in rows that are `pad` elements longer."""
    if not pad:
        return t
    wide = torch.empty(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    t = _TYPES[case["dtype"]]
    if case["op"] in ("embed", "embed_grad"):
        N, m, K, D = case["N"], case["m"], case["K"], case["D"]
        idx = _classes(N, m, K, g)
        s["idx"] = idx if m > 1 else idx[:, 0].contiguous()
        s["resp"] = None
        if case["weights"]:
            s["resp"] = torch.softmax(_randn(g, N, m) * 2.0, 1)
            s["resp"] = s["resp"] if m > 1 else torch.rand(N, generator=g, device="cuda")
        s["scale"] = 1.0 if case["weights"] else math.sqrt(D)
        if case["op"] == "embed" or case["weights"]:
            s["W"] = _rows_of(_randn(g, K, D, dtype=t).mul_(0.02), case["pad"])
        if case["op"] == "embed_grad":
            s["dY"] = _rows_of(_randn(g, N, D, dtype=t), case["pad"])
            s["dW"] = _randn(g, K, D) if case["add"] else None
        return s
    if case["op"] == "beam":
        B, w, K = case["B"], case["w"], case["K"]
        Z = torch.randn(B * w, K + case["pad"], generator=g, device="cuda").mul_(2.5)
        rows = torch.arange(B * w, device="cuda")
        for lift in (9.0, 8.0, 7.0, 5.0, 4.0):
            Z[rows, torch.randint(K, (B * w,), generator=g, device="cuda")] += lift
        s["scores"] = _randn(g, B, w).mul_(1.5).sub_(20.0).sort(1, descending=True).values
        s["ended"] = None
        if case["masks"]:
            cut = 0.5 * torch.rand(B * w, 1, generator=g, device="cuda")
            Z.masked_fill_(torch.rand(Z.shape, generator=g, device="cuda") < cut, -math.inf)
            s["ended"] = torch.rand(B, w, generator=g, device="cuda") < 0.15
            s["scores"][::7, 1:] = -math.inf  # searches that have just begun: one beam
        s["Z"] = Z.to(t)[:, :K]
        return s
    if case["op"] == "reorder":
        B, w = case["B"], case["w"]
        s["parent"] = torch.randint(w, (B, w), generator=g, device="cuda", dtype=torch.int32)
        s["lens"] = torch.randint(case["least"], case["most"] + 1, (B,), generator=g,
                                  device="cuda", dtype=torch.int32)
        s["states"] = [_randn(g, B * w, case["H"], case["T"], case["d"], dtype=t)
                       for _ in range(case["n"])]
        return s
    N, K, m, S = case["N"], case["K"], case["m"], case["S"]
    s["Z"] = (torch.randn(N, K, generator=g, device="cuda") * 1.5
              + torch.randn(K, generator=g, device="cuda")).to(t)
    s["mask"] = s["offsets"] = None
    if case["masks"]:
        s["mask"] = torch.rand(N, generator=g, device="cuda") < 0.9
    if S:  # packed sequences, rows behind the last one
        cuts = torch.rand(S, generator=g, device="cuda").sort().values
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts * (0.97 * N)]).int()
    s["idx"] = _largest(s["Z"].float(), m)[1].int()
    if case["op"] == "route_grad":
        s["dresp"] = _randn(g, N, m)
        S = max(S, 1)
        s["dbalance"] = torch.rand(S, generator=g, device="cuda").mul_(0.02 * N)
        s["dz"] = torch.rand(S, generator=g, device="cuda").mul_(0.001 * N)
        s["counts"], s["rows"] = _counts(s)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"embed": _run_embed, "embed_grad": _run_embed_grad, "beam": _run_beam,
            "reorder": _run_reorder, "balance": _run_balance,
            "route_grad": _run_route_grad}[state["op"]](state)


def _choices(s):
    """idx and resp as N x m; a choice of -1 has weight 0."""
    idx = s["idx"].view(s["N"], s["m"]).long()
    r = torch.ones_like(idx, dtype=torch.float32) if s["resp"] is None else s["resp"]
    return idx.clamp(min=0), r.view(idx.shape).masked_fill(idx < 0, 0.0)


def _run_embed(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        return G.gmm_embed(s["W"], s["idx"], s["resp"], scale=s["scale"])
    idx, r = _choices(s)
    return ((s["W"][idx].float() * r[:, :, None]).sum(1) * s["scale"]).to(s["W"].dtype)


def _run_embed_grad(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        dW, dresp = G.gmm_embed_backward(s["dY"], s["idx"], s["K"], s["resp"],
                                         W=s["W"] if s["weights"] else None, scale=s["scale"],
                                         out=s["dW"], accumulate=s["add"])
        return dict(dW=dW, dresp=dresp) if s["weights"] else dict(dW=dW)
    idx, r = _choices(s)
    dY = s["dY"].float() * s["scale"]
    terms = (dY[:, None] * r[:, :, None]).flatten(0, 1)
    if s["add"]:
        out = dict(dW=s["dW"].index_add_(0, idx.flatten(), terms))
    else:
        dW = torch.zeros(s["K"], s["D"], device=dY.device).index_add_(0, idx.flatten(), terms)
        out = dict(dW=dW.to(s["dY"].dtype))
    if s["weights"]:
        dots = (s["W"][idx].float() * dY[:, None]).sum(2)
        dots = dots.masked_fill(s["idx"].view(idx.shape) < 0, 0.0)
        out["dresp"] = dots.view(s["resp"].shape)
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
    return v, i.masked_fill(v == -math.inf, -1)


def _run_beam(s):
    B, w, m = s["B"], s["w"], s["m"]
    if own:
        from soft_clustering_em_b200 import gmm as G

        r = G.gmm_beam_select(s["Z"], s["scores"], m, ended=s["ended"], end_id=2,
                              scale=s["scale"])
        return dict(scores=r.scores, parent=r.parent, token=r.token)
    x = s["Z"].float()
    _, k = _largest(x * s["scale"], m)
    top = x.amax(1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    total = ((x - top) * s["scale"]).exp().sum(1, keepdim=True)
    # the candidates' scores lie close together: those in 64 bits
    v = (x.gather(1, k.clamp(min=0)).double() - top) * s["scale"] - total.double().log()
    v = v.masked_fill(k < 0, -math.inf).view(B, w, m) + s["scores"].double()[:, :, None]
    k = k.view(B, w, m)
    if s["ended"] is not None:
        first = torch.arange(m, device=x.device) == 0
        alone = s["scores"].double()[:, :, None].masked_fill(~first, -math.inf)
        v = torch.where(s["ended"][:, :, None], alone, v)
        k = k.masked_fill(s["ended"][:, :, None], 2)
    v, at = v.flatten(1).sort(dim=1, descending=True, stable=True)
    v, at = v[:, :m], at[:, :m]
    none = v == -math.inf
    return dict(scores=v.float(), parent=(at // m).int().masked_fill(none, -1),
                token=k.flatten(1).gather(1, at).int().masked_fill(none, -1))


def _run_reorder(s):
    B, w, T = s["B"], s["w"], s["T"]
    if own:
        from soft_clustering_em_b200 import gmm as G

        G.gmm_beam_reorder(s["states"], s["parent"], lens=s["lens"], dim=2)
        return s["states"]
    rows = (s["parent"] + torch.arange(B, device="cuda")[:, None] * w).view(-1)
    used = torch.arange(T, device="cuda") < s["lens"].repeat_interleave(w)[:, None]
    for t in s["states"]:
        t.copy_(torch.where(used[:, None, :, None], t[rows], t))
    return s["states"]


def _segments(s):
    """S x N: which rows count in which segment."""
    n = torch.arange(s["N"], device="cuda")
    live = s["Z"].float().amax(1) > -math.inf
    if s["mask"] is not None:
        live = live & s["mask"]
    if s["offsets"] is None:
        return live[None]
    o = s["offsets"][:, None]
    return (n >= o[:-1]) & (n < o[1:]) & live


def _counts(s):
    seg = _segments(s)
    S, K = seg.shape[0], s["K"]
    at = seg.int().argmax(0)[:, None] * K + s["idx"].clamp(min=0)
    one = (seg.any(0)[:, None] & (s["idx"] >= 0)).int()
    counts = torch.zeros(S * K, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, at.flatten().long(), one.flatten())
    return counts.view(S, K), seg.sum(1, dtype=torch.int32)


def _softmax(s):
    z = s["Z"].float()
    top = z.amax(1, keepdim=True)
    e = (z - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = e.sum(1, keepdim=True)
    return e / total, (top + total.log())[:, 0]


def _run_balance(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        r = G.gmm_route_loss(s["Z"], s["idx"], offsets=s["offsets"], mask=s["mask"])
        return dict(balance=r.balance, z=r.z, load=r.load, counts=r.counts, rows=r.rows)
    p, lse = _softmax(s)
    seg = _segments(s).float()
    counts, rows = _counts(s)
    L = rows.clamp(min=1).float()
    load = seg @ p / L[:, None]
    balance = (counts.float() * load).sum(1) * s["K"] / (s["m"] * L)
    return dict(balance=balance, z=seg @ lse.square() / L, load=load, counts=counts, rows=rows)


def _run_route_grad(s):
    if own:
        from soft_clustering_em_b200 import gmm as G

        return G.gmm_route_backward(s["Z"], s["idx"], s["dresp"], s["renorm"], s["counts"],
                                    s["rows"], s["dbalance"], s["dz"], offsets=s["offsets"],
                                    mask=s["mask"])
    p, lse = _softmax(s)
    seg = _segments(s).float()
    L = s["rows"].clamp(min=1).float()
    slope = s["counts"].float() * (s["dbalance"] * s["K"] / (s["m"] * L * L))[:, None]
    g = seg.T @ slope
    pull = (seg.T @ (2.0 * s["dz"] / L)) * lse
    i = s["idx"].long().clamp(min=0)
    d = s["dresp"].masked_fill(s["idx"] < 0, 0.0)
    q = p.gather(1, i).masked_fill(s["idx"] < 0, 0.0)
    if s["renorm"]:
        q = q / q.sum(1, keepdim=True)
        grad = p * (g - (p * g).sum(1, keepdim=True) + pull[:, None])
        grad.scatter_add_(1, i, q * (d - (q * d).sum(1, keepdim=True)))
    else:
        inner = (p * g).sum(1, keepdim=True) + (q * d).sum(1, keepdim=True)
        grad = p * (g - inner + pull[:, None])
        grad.scatter_add_(1, i, q * d)
    return grad.to(s["Z"].dtype)


# ------------------------------------------------------------------ the work of a pass
def work(case):
    b = _BYTES[case["dtype"]]
    if case["op"] in ("embed", "embed_grad"):
        N, m, K, D = case["N"], case["m"], case["K"], case["D"]
        named = _named(N, m, K)
        ids = 4.0 * N * m * (2 if case["weights"] else 1)
        if case["op"] == "embed":
            return dict(bytes=b * D * (named + N) + ids, flops=2.0 * N * m * D)
        bytes_ = b * N * D + ids + (2 * 4 * named * D if case["add"] else b * K * D)
        if case["weights"]:
            bytes_ += b * named * D + 4 * N * m
        return dict(bytes=bytes_, flops=(4.0 if case["weights"] else 2.0) * N * m * D)
    if case["op"] == "beam":
        rows = case["B"] * case["w"]
        return dict(bytes=1.0 * rows * case["K"] * b + 12 * case["B"] * case["m"],
                    flops=4.0 * rows * case["K"])
    if case["op"] == "reorder":
        w = case["w"]  # w - 1 beams move on average, from so many different ones:
        sources = w * (1.0 - (1.0 - 1.0 / w) ** (w - 1))
        used = 0.5 * (case["least"] + case["most"]) * case["H"] * case["d"] * b
        return dict(bytes=case["n"] * case["B"] * used * (w - 1 + sources), flops=0.0)
    N, K, m, S = case["N"], case["K"], case["m"], max(case["S"], 1)
    if case["op"] == "balance":
        return dict(bytes=1.0 * N * K * b + 4 * N * m + S * (8 * K + 12), flops=4.0 * N * K)
    return dict(bytes=2.0 * N * K * b + 8 * N * m + 4 * S * K, flops=8.0 * N * K)


def _named(N, m, K):
    """Different classes among N rows of _classes(), on average (by 1000 steps of the ranks)."""
    total, lo, logK = 0.0, 1.0, math.log(K + 1)
    for i in range(1, 1001):
        hi = (K + 1) ** (i / 1000)
        width = hi - lo  # about this many classes share a thousandth of the draws
        total += width * (1.0 - math.exp(-N * m / (1000 * width)))
        lo = hi
    return min(total, K, N * m)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_grad": _exact_embed_grad, "beam": _exact_beam,
            "reorder": _exact_reorder, "balance": _exact_balance,
            "route_grad": _exact_route_grad}[case["op"]](s)


def _exact_embed(s):
    W = torch.cat([s["W"].double(), torch.zeros(1, s["D"], dtype=torch.float64, device="cuda")])
    idx = s["idx"].view(s["N"], -1).long()
    y = torch.zeros(s["N"], s["D"], dtype=torch.float64, device="cuda")
    for j in range(s["m"]):  # (index -1 is the row of zeros)
        row = W[idx[:, j]]
        y += row if s["resp"] is None else row * s["resp"].view(idx.shape)[:, j:j + 1].double()
    return y * s["scale"]


def _exact_embed_grad(s):
    n, j = (s["idx"].view(s["N"], -1) >= 0).nonzero(as_tuple=True)
    k = s["idx"].view(s["N"], -1)[n, j].long()
    dY = s["dY"].double() * s["scale"]
    k, order = torch.sort(k, stable=True)
    terms = dY[n[order]]
    if s["resp"] is not None:
        r = s["resp"].view(s["N"], -1).double()
        terms *= r[n, j][order][:, None]
    lengths = torch.bincount(k, minlength=s["K"])
    dW = torch.segment_reduce(terms, "sum", lengths=lengths, initial=0.0)
    out = dict(dW=dW + s["dW"].double() if s["add"] else dW)
    if s["weights"]:
        dresp = torch.zeros_like(r)
        dresp[n, j] = torch.einsum("ad,ad->a", s["W"].double()[s["idx"].view(s["N"], -1)[n, j].long()],
                                   dY[n])
        out["dresp"] = dresp.view(s["resp"].shape)
    return out


def _exact_beam(s):
    B, w, m = s["B"], s["w"], s["m"]
    best = []
    for b in range(B):
        q = torch.log_softmax(s["Z"][b * w:(b + 1) * w].double() * s["scale"], 1)
        q = torch.where(q.isnan(), -math.inf, q) + s["scores"][b].double()[:, None]
        if s["ended"] is not None:
            alone = torch.full_like(q, -math.inf)
            alone[:, 2] = s["scores"][b].double()
            q = torch.where(s["ended"][b][:, None], alone, q)
        v = q.flatten().topk(min(m, q.numel())).values
        best.append(torch.nn.functional.pad(v, (0, m - len(v)), value=-math.inf))
    return dict(scores=torch.stack(best), parent=None, token=None)


def _exact_reorder(s):
    w, out = s["w"], []
    for t in s["states"]:
        t = t.double()
        now = t.clone()
        for b, n in enumerate(s["lens"].tolist()):
            group = t[b * w:(b + 1) * w]
            now[b * w:(b + 1) * w, :, :n] = group[s["parent"][b].long(), :, :n]
        out.append(now)
    return out


def _parts(s):
    """The rows that count of each segment."""
    o = [0, s["N"]] if s["offsets"] is None else s["offsets"].tolist()
    for lo, hi in zip(o[:-1], o[1:]):
        n = torch.arange(lo, hi, device="cuda")
        yield n if s["mask"] is None else n[s["mask"][lo:hi]]


def _exact_balance(s):
    out = dict(balance=[], z=[], load=[])
    for n in _parts(s):
        z = s["Z"][n].double()
        L = max(len(n), 1)
        f = torch.bincount(s["idx"][n].flatten().long(), minlength=s["K"]).double() / (s["m"] * L)
        P = torch.softmax(z, 1).sum(0) / L
        out["load"].append(P)
        out["balance"].append(s["K"] * torch.dot(f, P))
        out["z"].append((torch.logsumexp(z, 1) ** 2).sum() / L)
    return dict({k: torch.stack(v) for k, v in out.items()}, counts=None, rows=None)


def _exact_route_grad(s):
    Z = s["Z"].double().requires_grad_()
    p = torch.softmax(Z, 1)
    chosen = p.gather(1, s["idx"].long())
    resp = chosen / chosen.sum(1, keepdim=True) if s["renorm"] else chosen
    value = (resp * s["dresp"].double()).sum()
    lse = torch.logsumexp(Z, 1)
    for i, n in enumerate(_parts(s)):
        if len(n):
            f = s["counts"][i].double() / (s["m"] * len(n))
            value = value + s["dbalance"][i].double() * s["K"] * torch.dot(f, p[n].mean(0))
            value = value + s["dz"][i].double() * (lse[n] ** 2).mean()
    return torch.autograd.grad(value, Z)[0]
