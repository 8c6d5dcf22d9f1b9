"""Timed cases of the softmax head, codebook and gradient-clipping operators.

Each case is one call (or one training step's calls) with the sizes it runs at
in use; `run` computes it either with elementary torch operations in 32 bits
(own = False) or with the library's calls (own = True), `exact` in 64 bits.

  xent     softmax cross entropy of rows under a linear head (V classes, no
           logits kept): "score" is the loss alone, "step" the loss and the
           gradients of the rows, the head and the bias
  lookup   rows rebuilt from codes: out_i = scale * sum_j w_ij T[idx_ij]
  scatter  the gradient of that lookup: the table's, and the weights' where given
  clip     the norm over all gradients and the gradients scaled by it
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _g():
    import soft_clustering_em_amd as g
    return g


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's log-probability under a vocabulary head (serving, batch 1)
        dict(name="score_one", op="xent", grad=False, N=1, D=2048, V=32768, dtype="bf16", bias=False, pad=0, ignored=0.0),
        # log-probabilities of a ragged batch of half rows under a head of odd size
        dict(name="score_batch", op="xent", grad=False, N=1000, D=1000, V=50001, dtype="f16", bias=True, pad=0,
             ignored=0.05),
        # a classifier over the lists of the coarse quantizer (D = 128, 4096 lists), one training step
        dict(name="router_step", op="xent", grad=True, N=262144, D=128, V=4096, dtype="bf16", bias=True, pad=0,
             ignored=0.0),
        # the posterior head of the 256-component diagonal workload (1M x 64, float32), one training step
        dict(name="posterior_step", op="xent", grad=True, N=1000000, D=64, V=256, dtype="f32", bias=True, pad=0,
             ignored=0.0),
        # a vocabulary head over a batch of 4096 tokens, one training step
        dict(name="vocab_step", op="xent", grad=True, N=4096, D=4096, V=65536, dtype="bf16", bias=False, pad=0,
             ignored=0.02),
        # odd sizes, rows of a wider array, padded labels
        dict(name="odd_step", op="xent", grad=True, N=777, D=515, V=10007, dtype="f16", bias=True, pad=13, ignored=0.3),
        # one token's embedding (serving, batch 1)
        dict(name="embed_one", op="lookup", N=1, m=1, D=4096, K=131072, dtype="bf16", weighted=False, scale=64.0),
        # rows rebuilt from the top-4 multi-assignment of the coarse quantizer
        dict(name="rebuild", op="lookup", N=1000000, m=4, D=128, K=4096, dtype="f32", weighted=True, scale=1.0),
        # the embedding gradient of a batch of tokens (frequencies fall with the rank)
        dict(name="embed_grad", op="scatter", N=32768, m=1, D=2048, K=65536, dtype="bf16", weighted=False, scale=1.0),
        # the codebook's and the responsibilities' gradients behind a rebuilt batch
        dict(name="rebuild_grad", op="scatter", N=262144, m=4, D=128, K=4096, dtype="f32", weighted=True, scale=1.0),
        # the gradients of a small head: many small tensors of odd sizes
        dict(name="clip_small", op="clip", tensors=24, smallest=1, largest=20000, dtype="f32", max_norm=1.0),
        # the gradients of a large model: tensors from a bias to a vocabulary matrix, two types
        dict(name="clip_large", op="clip", tensors=48, smallest=2048, largest=67108864, dtype="mixed", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["xent", "xent", "lookup", "scatter", "clip"])
    if op == "xent":
        while True:
            N, D, V = _log(rng, 1, 1000000), _log(rng, 8, 4096), _log(rng, 2, 131072)
            if rng.random() < 0.5:
                D = (D + 7) // 8 * 8
            if N * D * V <= 4096 * 4096 * 65536 and N * V <= 1 << 30 and N * D <= 1 << 28:
                break
        return dict(op=op, grad=rng.random() < 0.6, N=N, D=D, V=V, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    bias=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 13]), ignored=rng.choice([0.0, 0.05, 0.5]))
    if op in ("lookup", "scatter"):
        while True:
            N, m, D, K = _log(rng, 1, 1000000), rng.choice([1, 1, 2, 3, 4, 8, 16]), _log(rng, 8, 8192), _log(rng, 1, 131072)
            if N * D <= 1 << 27 and N * m * D <= 1 << 28 and K * D <= 1 << 28:
                break
        return dict(op=op, N=N, m=m, D=D, K=K, dtype=rng.choice(["bf16", "f16", "f32"]),
                    weighted=m > 1 or rng.random() < 0.3, scale=rng.choice([1.0, 0.5, 11.3]))
    return dict(op=op, tensors=_log(rng, 1, 60), smallest=1, largest=_log(rng, 16, 4000000),
                dtype=rng.choice(["f32", "bf16", "f16", "mixed"]), max_norm=rng.choice([0.1, 1.0, 1e6]))


def _clip_sizes(case):
    """Sizes from smallest to largest, evenly spaced in the logarithm."""
    n, lo, hi = case["tensors"], case["smallest"], case["largest"]
    return [max(1, int(round(lo * (hi / lo) ** (i / max(1, n - 1))))) for i in range(n)]


def _clip_types(case):
    n = case["tensors"]
    if case["dtype"] == "mixed":
        return [torch.float32 if i % 4 == 0 else torch.bfloat16 for i in range(n)]
    return [DTYPES[case["dtype"]]] * n


# ---------------------------------------------------------------- inputs

def _codes(case, gen):
    """Codes as a top-m assignment writes them: 1..m distinct leading codes a row,
    -1 behind them, larger responsibilities first; with m = 1, codes whose
    frequency falls as 1 / rank."""
    N, m, K = case["N"], case["m"], case["K"]
    u = torch.rand(N, generator=gen, device="cuda", dtype=torch.float64)
    first = (torch.exp(u * math.log(K + 1.0)) - 1.0).long().clamp_(0, K - 1)
    step = 1 + torch.randint(0, max(1, (K - 1) // max(1, m)), (N, 1), generator=gen, device="cuda")
    idx = (first[:, None] + step * torch.arange(m, device="cuda")) % K
    keep = torch.randint(1, m + 1, (N, 1), generator=gen, device="cuda").clamp_max(K)
    behind = torch.arange(m, device="cuda") >= keep
    idx = idx.masked_fill(behind, -1).to(torch.int32).contiguous()
    weights = None
    if case["weighted"]:
        r = torch.rand(N, m, generator=gen, device="cuda").add_(0.05).masked_fill_(behind, 0.0)
        weights = (r / r.sum(1, keepdim=True)).sort(dim=1, descending=True).values.contiguous()
    return idx, weights


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = dict(case=case)
    if case["op"] == "xent":
        N, D, V, dt = case["N"], case["D"], case["V"], DTYPES[case["dtype"]]
        st["X"] = torch.randn(N, D + case["pad"], generator=gen, device="cuda").to(dt)[:, :D]
        st["W"] = (torch.randn(V, D, generator=gen, device="cuda") * (2.0 / math.sqrt(D))).to(dt)
        st["bias"] = torch.randn(V, generator=gen, device="cuda") if case["bias"] else None
        y = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
        drop = torch.rand(N, generator=gen, device="cuda") < case["ignored"]
        st["labels"] = y.masked_fill(drop, -1)
        # the mean over the labelled rows; half rows carry a loss scale that keeps the
        # gradients of rows and head inside their range
        n = (~drop).sum().clamp_min(1)
        scale = 2.0 ** round(math.log2(N) / 2) if dt == torch.float16 else 1.0
        st["gloss"] = torch.full((N,), scale, device="cuda") / n
    elif case["op"] in ("lookup", "scatter"):
        dt = DTYPES[case["dtype"]]
        st["idx"], st["weights"] = _codes(case, gen)
        if case["op"] == "lookup" or case["weighted"]:
            st["table"] = torch.randn(case["K"], case["D"], generator=gen, device="cuda").to(dt)
        if case["op"] == "scatter":
            st["dout"] = torch.randn(case["N"], case["D"], generator=gen, device="cuda").to(dt)
    else:
        st["grads"] = [torch.randn(n, generator=gen, device="cuda").mul_(1e-2).to(t)
                       for n, t in zip(_clip_sizes(case), _clip_types(case))]
        st["out"] = [torch.empty_like(t) for t in st["grads"]]
    return st


# ---------------------------------------------------------------- one pass

def _plain_xent(st):
    X, W, y = st["X"].float(), st["W"].float(), st["labels"].long()
    logits = X @ W.t()
    if st["bias"] is not None:
        logits = logits + st["bias"]
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    live = y >= 0
    rows = torch.arange(y.numel(), device=y.device)
    at = y.clamp_min(0)
    loss = torch.where(live, lse - logits[rows, at], torch.zeros_like(lse))
    if not st["case"]["grad"]:
        return loss, lse
    G = e / total
    G[rows, at] -= 1.0
    G = G * torch.where(live, st["gloss"], torch.zeros_like(st["gloss"]))[:, None]
    dX = (G @ W).to(st["X"].dtype)
    if X.dtype != st["X"].dtype:
        dW = (G.t() @ X).to(st["W"].dtype)
    else:
        # float32 gradients of the head sum up to a million rows: pieces of
        # 8192 rows in 32 bits, joined in 64, keep their last digits
        pad = -X.shape[0] % 8192 if X.shape[0] > 8192 else 0
        piece = min(X.shape[0], 8192)
        Gp, Xp = (torch.nn.functional.pad(t, (0, 0, 0, pad)).unflatten(0, (-1, piece)) for t in (G, X))
        dW = torch.bmm(Gp.transpose(1, 2), Xp).sum(dim=0, dtype=torch.float64).float()
    return (loss, lse, dX, dW) + ((G.sum(dim=0),) if st["bias"] is not None else ())


def _plain_weights(st):
    """float32 weight of every slot: 0 behind a row's codes, and there code 0."""
    live = st["idx"] >= 0
    w = live.float() if st["weights"] is None else torch.where(live, st["weights"], torch.zeros_like(st["weights"]))
    return st["idx"].clamp_min(0).long(), w, live


def _plain_lookup(st):
    at, w, _ = _plain_weights(st)
    return (st["case"]["scale"] * (w[:, :, None] * st["table"][at].float()).sum(dim=1)).to(st["table"].dtype)


def _plain_scatter(st):
    at, w, live = _plain_weights(st)
    s, dout = st["case"]["scale"], st["dout"].float()
    acc = torch.zeros(st["case"]["K"], dout.shape[1], device=at.device)
    acc.index_add_(0, at.flatten(), (w[:, :, None] * dout[:, None, :]).flatten(0, 1))
    dtable = (s * acc).to(st["dout"].dtype)
    if st["weights"] is None:
        return dtable
    dw = s * (dout[:, None, :] * st["table"][at].float()).sum(dim=2)
    return dtable, torch.where(live, dw, torch.zeros_like(dw))


def _plain_clip(st):
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for t in st["grads"]:
        total = total + t.float().square().sum(dtype=torch.float64)
    norm = torch.sqrt(total)
    c = (st["case"]["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
    return [(c * t.float()).to(t.dtype) for t in st["grads"]] + [norm.float().reshape(1)]


def run(st):
    case = st["case"]
    if not own:
        plain = {"xent": _plain_xent, "lookup": _plain_lookup, "scatter": _plain_scatter, "clip": _plain_clip}
        return plain[case["op"]](st)
    g = _g()
    if case["op"] == "xent":
        loss, lse = g.gmm_softmax_xent(st["X"], st["W"], st["labels"], bias=st["bias"])
        if not case["grad"]:
            return loss, lse
        dX, dW, db = g.gmm_softmax_xent_grad(st["X"], st["W"], st["labels"], lse, gloss=st["gloss"], bias=st["bias"])
        return (loss, lse, dX, dW) + ((db,) if db is not None else ())
    if case["op"] == "lookup":
        return g.gmm_codebook_lookup(st["table"], st["idx"], weights=st["weights"], scale=case["scale"])
    if case["op"] == "scatter":
        dtable, dweights = g.gmm_codebook_lookup_grad(st["dout"], st["idx"], case["K"], table=st.get("table"),
                                                      weights=st["weights"], scale=case["scale"])
        return dtable if dweights is None else (dtable, dweights)
    norm = g.gmm_clip_grad_norm(st["grads"], case["max_norm"], out=st["out"])
    return st["out"] + [norm]


# ---------------------------------------------------------------- what a pass needs

def work(case):
    if case["op"] == "xent":
        N, D, V, e = case["N"], case["D"], case["V"], 4 if case["dtype"] == "f32" else 2
        bias = 4 * V if case["bias"] else 0
        b = e * (N * D + V * D) + bias + 4 * N + 8 * N
        if not case["grad"]:
            return {"bytes": b, "flops": 2 * N * V * D}
        return {"bytes": b + e * (N * D + V * D) + bias + 4 * N, "flops": 6 * N * V * D}
    if case["op"] in ("lookup", "scatter"):
        N, m, D, K, e = case["N"], case["m"], case["D"], case["K"], 4 if case["dtype"] == "f32" else 2
        entries = N * (m + 1) // 2  # a row keeps 1..m codes, evenly
        codes = 4 * N * m * (2 if case["weighted"] else 1)
        touched = min(entries, K)
        if case["op"] == "lookup":
            return {"bytes": codes + e * D * (touched + N), "flops": 2 * entries * D}
        b = codes + e * D * (N + K)
        if case["weighted"]:
            b += e * D * touched + 4 * N * m
        return {"bytes": b, "flops": (4 if case["weighted"] else 1) * entries * D}
    n = sum(s * (4 if t == torch.float32 else 2) for s, t in zip(_clip_sizes(case), _clip_types(case)))
    return {"bytes": 2 * n, "flops": 3 * sum(_clip_sizes(case))}


# ---------------------------------------------------------------- 64 bits

def _exact_xent(st):
    """Rows in pieces; log-softmax through torch's float64 logsumexp."""
    X, W, y = st["X"].double(), st["W"].double(), st["labels"]
    N, V = X.shape[0], W.shape[0]
    b = None if st["bias"] is None else st["bias"].double()
    loss, lse = (torch.empty(N, device="cuda", dtype=torch.float64) for _ in range(2))
    grad = st["case"]["grad"]
    dX, dW = (torch.zeros_like(X), torch.zeros_like(W)) if grad else (None, None)
    db = torch.zeros(V, device="cuda", dtype=torch.float64)
    piece = max(1, (1 << 28) // V)
    for r0 in range(0, N, piece):
        part = slice(r0, min(N, r0 + piece))
        L = torch.mm(X[part], W.t())
        if b is not None:
            L += b
        z = torch.logsumexp(L, dim=1)
        lse[part] = z
        on = (y[part] >= 0).double()
        label = y[part].clamp(min=0).long().unsqueeze(1)
        loss[part] = on * (z - L.gather(1, label)[:, 0])
        if grad:
            P = L.sub_(z[:, None]).exp_()
            P.scatter_add_(1, label, torch.full_like(label, -1, dtype=torch.float64))
            P *= (on * st["gloss"][part].double())[:, None]
            dX[part] = torch.mm(P, W)
            dW += torch.mm(P.t(), X[part])
            db += P.sum(0)
    if not grad:
        return loss, lse
    return (loss, lse, dX, dW) + ((db,) if b is not None else ())


def _exact_entries(st):
    """The (row, slot, code, weight) of every kept code."""
    row, slot = torch.nonzero(st["idx"] >= 0, as_tuple=True)
    code = st["idx"][row, slot].long()
    w = torch.ones(row.numel(), device="cuda", dtype=torch.float64) if st["weights"] is None \
        else st["weights"][row, slot].double()
    return row, slot, code, w


def _exact_codes(st):
    row, slot, code, w = _exact_entries(st)
    case = st["case"]
    N, D, K, s = case["N"], case["D"], case["K"], float(case["scale"])
    lookup = case["op"] == "lookup"
    res = torch.zeros(N if lookup else K, D, device="cuda", dtype=torch.float64)
    dw = torch.zeros(N, case["m"], device="cuda", dtype=torch.float64)
    piece = max(1, (1 << 27) // D)
    for e0 in range(0, row.numel(), piece):
        r, j, k, we = (t[e0:e0 + piece] for t in (row, slot, code, w))
        if lookup:
            res.index_add_(0, r, (s * we)[:, None] * st["table"][k].double())
            continue
        d = st["dout"][r].double()
        if st["weights"] is not None:
            dw[r, j] = s * (d * st["table"][k].double()).sum(1)
        res.index_add_(0, k, d.mul_((s * we)[:, None]))
    if lookup or st["weights"] is None:
        return res
    return res, dw


def _exact_clip(st):
    squares = [(t.double() ** 2).sum() for t in st["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    c = min(1.0, st["case"]["max_norm"] / (float(norm) + 1e-6))
    return [t.double() * c for t in st["grads"]] + [norm.reshape(1)]


def exact(case, seed):
    st = prepare(case, seed)
    return {"xent": _exact_xent, "lookup": _exact_codes, "scatter": _exact_codes, "clip": _exact_clip}[case["op"]](st)
