"""Timed cases of the layer norm, routing, AdamW and sampling operators.

Each case is one call (or one training step's calls) with the sizes it runs at
in use; `run` computes it either with elementary torch operations (own = False)
or with the library's calls (own = True), `exact` in 64 bits.

  norm    layer norm of rows: "grad" adds the gradients of rows, scale and shift
  route   scores of experts turned into the top-m codes and weights that a
          codebook lookup reads: "grad" adds the scores' gradient
  adamw   one AdamW step over many tensors, gradients clipped by a given norm,
          states of 32 bits, or of 8 with a scale for every 256 values
  sample  one token a row from logits with temperature, min-p, top-k and top-p,
          from one given uniform number a row
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
BLOCK = 256  # values under one scale of an 8-bit state
TOP = float(torch.finfo(torch.float32).max)
ADAMW = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_norm=1.0, seed=1234)


def _g():
    import soft_clustering_em_amd as g
    return g


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden row (serving, batch 1)
        dict(name="norm_one", op="norm", grad=False, N=1, D=4096, dtype="bf16", pad=0),
        # the rows of an embedding batch (32768 x 2048), one training step
        dict(name="norm_step", op="norm", grad=True, N=32768, D=2048, dtype="bf16", pad=0),
        # the rows of the 256-component diagonal workload (1M x 64), one training step
        dict(name="norm_narrow", op="norm", grad=True, N=1000000, D=64, dtype="f32", pad=0),
        # one token routed to 8 of 256 experts (serving, batch 1)
        dict(name="route_one", op="route", grad=False, N=1, E=256, m=8, score="sigmoid", bias=True, groups=8, keep=4,
             top=2, renorm=True, dtype="f32", masked=0.0),
        # a batch of tokens routed to 8 of 256 experts in the 4 best of 8 groups, balanced by a bias
        dict(name="route_batch", op="route", grad=False, N=65536, E=256, m=8, score="sigmoid", bias=True, groups=8, keep=4,
             top=2, renorm=True, dtype="f32", masked=0.0),
        # a training step of a softmax router over an odd number of experts, some of them switched off
        dict(name="route_step", op="route", grad=True, N=100000, E=60, m=4, score="softmax", bias=False, groups=1, keep=1,
             top=1, renorm=True, dtype="bf16", masked=0.05),
        # the step of a small head: tensors of odd sizes, a single value among them
        dict(name="adamw_small", op="adamw", tensors=12, smallest=1, largest=20000, dtype="f32", bits=32, copies=False),
        # a large model's step: float32 weights with bf16 copies, bf16 gradients, float32 states
        dict(name="adamw_large", op="adamw", tensors=12, smallest=2048, largest=67108864, dtype="mixed", bits=32, copies=True),
        # the same weights with states of 8 bits
        dict(name="adamw_8bit", op="adamw", tensors=12, smallest=2048, largest=67108864, dtype="mixed", bits=8, copies=False),
        # one token's sampling over a vocabulary (serving, batch 1)
        dict(name="sample_one", op="sample", N=1, V=131072, dtype="bf16", temperature=0.8, top_k=50, top_p=0.9, min_p=0.0,
             mixed=False),
        # a serving batch over a vocabulary, nucleus sampling
        dict(name="sample_batch", op="sample", N=256, V=131072, dtype="bf16", temperature=0.7, top_k=0, top_p=0.9, min_p=0.0,
             mixed=False),
        # requests with settings of their own (some greedy, some unfiltered) over an odd vocabulary
        dict(name="sample_mixed", op="sample", N=77, V=50001, dtype="f32", temperature=1.0, top_k=40, top_p=0.95, min_p=0.05,
             mixed=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "adamw", "sample"])
    if op == "norm":
        while True:
            N, D = _log(rng, 1, 1000000), _log(rng, 8, 16384)
            if rng.random() < 0.5:
                D = (D + 7) // 8 * 8
            if N * D <= 1 << 26:
                break
        return dict(op=op, grad=rng.random() < 0.6, N=N, D=D, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    pad=rng.choice([0, 0, 8, 13]))
    if op == "route":
        while True:
            groups = rng.choice([1, 1, 1, 2, 4, 8])
            E = groups * _log(rng, 2, 512 // groups)
            N, m = _log(rng, 1, 262144), rng.choice([1, 2, 4, 6, 8, 16])
            keep = rng.randint(1, groups)
            if N * E <= 1 << 24 and m <= keep * (E // groups):
                break
        return dict(op=op, grad=rng.random() < 0.5, N=N, E=E, m=m, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    dtype=rng.choice(["f32", "bf16", "f16"]), masked=rng.choice([0.0, 0.0, 0.1]))
    if op == "adamw":
        return dict(op=op, tensors=rng.randint(1, 12), smallest=1, largest=_log(rng, 16, 4000000),
                    dtype=rng.choice(["f32", "bf16", "f16", "mixed"]), bits=rng.choice([32, 8]), copies=False)
    while True:
        N, V = _log(rng, 1, 1024), _log(rng, 2, 262144)
        if N * V <= 1 << 25:
            break
    return dict(op=op, N=N, V=V, dtype=rng.choice(["bf16", "f16", "f32"]), temperature=rng.choice([0.5, 1.0, 1.3]),
                top_k=rng.choice([0, 0, 1, 20, 200]), top_p=rng.choice([1.0, 0.5, 0.9, 0.99]),
                min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.3)


def _sizes(case):
    """Sizes from smallest to largest, evenly spaced in the logarithm."""
    n, lo, hi = case["tensors"], case["smallest"], case["largest"]
    return [max(1, int(round(lo * (hi / lo) ** (i / max(1, n - 1))))) for i in range(n)]


def _types(case):
    """(weight, gradient) types of every tensor; mixed: float32 weights, most gradients bf16."""
    n = case["tensors"]
    if case["dtype"] == "mixed":
        return [("f32", "f32" if i % 4 == 0 else "bf16") for i in range(n)]
    return [(case["dtype"], case["dtype"])] * n


# ---------------------------------------------------------------- inputs

def _quantised(t):
    """(e4m3 values, scale of every block) of a float32 vector."""
    n = t.numel()
    b = torch.nn.functional.pad(t, (0, -n % BLOCK)).view(-1, BLOCK)
    s = b.abs().amax(1) / 448.0
    q = (b / s.clamp_min(1e-30)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(-1)[:n].clone(), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    st = dict(case=case)
    if case["op"] == "norm":
        N, D, dt = case["N"], case["D"], DTYPES[case["dtype"]]
        # rows with means and spreads of their own
        st["X"] = (rand(N, D + case["pad"]) * (0.5 + torch.rand(N, 1, generator=gen, device="cuda")) + 0.3 * rand(N, 1)).to(dt)[:, :D]
        st["gamma"], st["beta"] = (1.0 + 0.1 * rand(D)).to(dt), (0.1 * rand(D)).to(dt)
        if case["grad"]:
            st["dout"] = rand(N, D).to(dt)
    elif case["op"] == "route":
        N, E, m = case["N"], case["E"], case["m"]
        logits = 1.5 * rand(N, E)
        off = torch.rand(N, E, generator=gen, device="cuda") < case["masked"]
        st["logits"] = logits.masked_fill_(off, -math.inf).to(DTYPES[case["dtype"]])
        st["bias"] = 0.05 * rand(E) if case["bias"] else None
        if case["grad"]:
            st["dweights"] = rand(N, m)
            # the balance loss's gradient, one value an expert
            st["dscores"] = 0.01 * rand(E)
    elif case["op"] == "adamw":
        st["step"] = 100
        st["p"], st["g"], st["m"], st["v"], st["ms"], st["vs"], st["copy"] = ([] for _ in range(7))
        for n, (tp, tg) in zip(_sizes(case), _types(case)):
            st["p"].append((0.02 * rand(n)).to(DTYPES[tp]))
            st["g"].append((1e-3 * rand(n)).to(DTYPES[tg]))
            m, v = 1e-3 * rand(n), (1e-3 * rand(n)).square_() + 1e-8
            if case["bits"] == 8:
                for name, t in (("m", m), ("v", v.sqrt())):
                    q, s = _quantised(t)
                    st[name].append(q)
                    st[name + "s"].append(s)
            else:
                st["m"].append(m)
                st["v"].append(v)
            if case["copies"]:
                st["copy"].append(torch.empty(n, device="cuda", dtype=torch.bfloat16))
        # the norm that gmm_clip_grad_norm leaves beside the gradients
        st["norm"] = torch.tensor([math.sqrt(sum(_sizes(case))) * 1e-3], device="cuda")
    else:
        N, V = case["N"], case["V"]
        st["logits"] = (2.5 * rand(N, V)).to(DTYPES[case["dtype"]])
        st["u"] = torch.rand(N, generator=gen, device="cuda")
        one = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
        for k, t in one.items():
            st[k] = case[k]
            if case["mixed"]:
                # a third of the requests without the filter, and some greedy ones
                off = dict(temperature=0.0, top_k=0, top_p=1.0, min_p=0.0)[k]
                third = torch.arange(N, device="cuda") % 3 == list(one).index(k) % 3
                st[k] = torch.full((N,), case[k], dtype=t, device="cuda").masked_fill_(third, off)
    return st


# ---------------------------------------------------------------- one pass

def _plain_norm(st):
    X, D = st["X"].float(), st["case"]["D"]
    gamma, beta = st["gamma"].float(), st["beta"].float()
    mean = X.sum(1) / D
    d = X - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / D + EPS)
    xh = d * rstd[:, None]
    out = (xh * gamma + beta).to(st["X"].dtype)
    if not st["case"]["grad"]:
        return out, mean, rstd
    dout = st["dout"].float()
    q = dout * gamma
    a, b = q.sum(1, keepdim=True) / D, (q * xh).sum(1, keepdim=True) / D
    dX = (rstd[:, None] * (q - a - xh * b)).to(st["X"].dtype)
    return out, mean, rstd, dX, (dout * xh).sum(0), dout.sum(0)


def _plain_scores(st):
    """64-bit scores s of every expert, 0 for those switched off, and which are on."""
    l = st["logits"].double()  # noqa: E741
    live = l > -math.inf
    l = torch.where(live, l, torch.full_like(l, -math.inf)).clamp_max(TOP)  # noqa: E741
    if st["case"]["score"] == "sigmoid":
        return l, torch.where(live, 1.0 / (1.0 + torch.exp(-l)), torch.zeros_like(l)), live
    top = l.max(1, keepdim=True).values.clamp_min(-TOP)
    e = torch.exp(l - top)
    return l, e / e.sum(1, keepdim=True).clamp_min(1e-300), live


def _plain_route(st):
    c = st["case"]
    N, E, m, G = c["N"], c["E"], c["m"], c["groups"]
    l, s, live = _plain_scores(st)  # noqa: E741
    none = torch.full_like(l, -math.inf)
    # without a bias the order of the scores is the order of the logits
    t = l if st["bias"] is None and (G == 1 or c["top"] == 1) else s + (0.0 if st["bias"] is None else st["bias"].double())
    t = torch.where(live, t, none)
    if G > 1:
        best = t.view(N, G, E // G).sort(dim=2, descending=True).values[:, :, :min(c["top"], E // G)]
        on = best > -math.inf
        score = torch.where(on[:, :, 0], torch.where(on, best, torch.zeros_like(best)).sum(2), none[:, :G])
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(N, G, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        t = torch.where(kept[:, :, None], t.view(N, G, E // G), none.view(N, G, E // G)).view(N, E)
        if st["bias"] is None and c["top"] == 2:
            t = torch.where(t > -math.inf, l, none)
    value, at = t.sort(dim=1, descending=True, stable=True)
    on, at = value[:, :m] > -math.inf, at[:, :m]
    idx = torch.where(on, at, torch.full_like(at, -1)).to(torch.int32)
    sel = torch.where(on, s.gather(1, at), torch.zeros_like(s[:, :m]))
    total = sel.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(sel[:, :1])
    q = sel / total.clamp_min(1e-300)
    weights = (2.5 * q).float()
    if not c["grad"]:
        return idx, weights
    # softmax: ds_e / dl_f = s_e ([e = f] - s_f); sigmoid: s (1 - s); renormalised: q_j = s_j / total
    dq = torch.where(on, 2.5 * st["dweights"].double(), torch.zeros_like(q))
    if c["renorm"]:
        dq = (dq - (dq * q).sum(1, keepdim=True)) / total.clamp_min(1e-300)
    ds = st["dscores"].double() + torch.zeros_like(s).scatter_add_(1, at, dq)
    if c["score"] == "softmax":
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    else:
        dl = ds * s * (1.0 / (1.0 + torch.exp(l)))
    return idx, weights, torch.where(live, dl, torch.zeros_like(dl)).to(st["logits"].dtype)


def _mix(x):
    """The library's 32-bit mixing function, in 64-bit integers."""
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _dither(n, j, step, seed):
    """16-bit numbers for the first and the second moment of every value of tensor j."""
    i = torch.arange(n, device="cuda")
    key = _mix(_mix(torch.tensor((seed + 0x9E3779B1 * step) & 0xFFFFFFFF, device="cuda")) ^ j)
    h = _mix((_mix((key + i // BLOCK) & 0xFFFFFFFF) + (i % BLOCK) * 0x9E3779B1) & 0xFFFFFFFF)
    return h >> 16, h & 0xFFFF


def _to_8bit(t, d, q, s, floor):
    """t into e4m3 values q and scales s, rounded up with the probability that the 16-bit numbers d give it."""
    n = t.numel()
    b = torch.nn.functional.pad(t, (0, -n % BLOCK)).view(-1, BLOCK)
    top = b.abs().amax(1)
    s.copy_(torch.where(top < 2.0 ** -100, torch.zeros_like(top), top / 448.0))
    inv = torch.where(top < 2.0 ** -100, torch.zeros_like(top), 448.0 / top)
    x = (b * inv[:, None]).view(-1)[:n]
    a = x.abs().clamp_max(448.0)
    bits = a.view(torch.int32) + (d << 4).int()
    normal = (bits & -0x100000).view(torch.float32)
    small = torch.floor(a * 512.0 + d.float() / 65536.0) / 512.0
    r = torch.where(a < 2.0 ** -6, small, normal)
    if floor:  # a second moment that is there does not vanish
        r = torch.where(x > 0.0, r.clamp_min(2.0 ** -9), r)
    q.copy_(torch.where(x < 0.0, -r, r).to(torch.float8_e4m3fn))


def _plain_adamw(st):
    c, o = st["case"], ADAMW
    (b1, b2), step = o["betas"], st["step"]
    clip = (o["max_norm"] / (st["norm"].double() + 1e-6)).clamp_max(1.0).float()
    alpha = o["lr"] / (1.0 - b1 ** step)
    root = 1.0 / math.sqrt(1.0 - b2 ** step)
    for j, (p, g) in enumerate(zip(st["p"], st["g"])):
        g = clip * g.float()
        m, v = st["m"][j], st["v"][j]
        if c["bits"] == 8:
            m = m.float() * st["ms"][j].repeat_interleave(BLOCK)[:m.numel()]
            r = v.float() * st["vs"][j].repeat_interleave(BLOCK)[:v.numel()]
            v = r * r
        m = b1 * m + (1.0 - b1) * g
        v = b2 * v + (1.0 - b2) * (g * g)
        r = torch.sqrt(v)
        new = p.float() * (1.0 - o["lr"] * o["weight_decay"]) - alpha * (m / (r * root + o["eps"]))
        p.copy_(new)
        if c["copies"]:
            st["copy"][j].copy_(new)
        if c["bits"] == 8:
            dm, dv = _dither(m.numel(), j, step, o["seed"])
            _to_8bit(m, dm, st["m"][j], st["ms"][j], False)
            _to_8bit(r, dv, st["v"][j], st["vs"][j], True)
        else:
            st["m"][j].copy_(m)
            st["v"][j].copy_(v)
    st["step"] += 1
    return st["p"], st["m"], st["v"], st["ms"], st["vs"], st["copy"]


def _per_row(st, name, dtype):
    """A setting as a column, one value a row."""
    v, N = st[name], st["case"]["N"]
    return v.to(dtype)[:, None] if isinstance(v, torch.Tensor) else torch.full((N, 1), v, dtype=dtype, device="cuda")


def _plain_sample(st):
    V = st["case"]["V"]
    l = st["logits"].double()  # noqa: E741
    T, k = _per_row(st, "temperature", torch.float64), _per_row(st, "top_k", torch.int64)
    top_p, min_p = _per_row(st, "top_p", torch.float64), _per_row(st, "min_p", torch.float64)
    k = torch.where((k <= 0) | (k > V), torch.full_like(k, V), k)
    k = torch.where(T > 0.0, k, torch.ones_like(k))
    T = torch.where(T > 0.0, T, torch.ones_like(T))
    l, order = l.sort(dim=1, descending=True, stable=True)  # noqa: E741
    w = torch.exp((l - l[:, :1]) / T)
    w = torch.where((torch.arange(V, device="cuda") < k) & (w >= min_p.clamp(0.0, 1.0)), w, torch.zeros_like(w))
    # top-p over what top-k leaves: the shortest prefix that reaches the share
    within = torch.exp((l - l[:, :1]) / T) * (torch.arange(V, device="cuda") < k)
    before = within.cumsum(1) - within
    cut = (top_p >= 1.0) | (before < top_p * within.sum(1, keepdim=True))
    cut[:, 0] = True
    w = torch.where(cut, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order, w)
    total = w.sum(1)
    run_ = w.cumsum(1)
    hit = (run_ > (st["u"].double() * total)[:, None]) & (w > 0.0)
    token = hit.to(torch.uint8).argmax(1)
    return token.to(torch.int32), torch.log(w.gather(1, token[:, None])[:, 0] / total).float()


def run(st):
    case = st["case"]
    if not own:
        plain = {"norm": _plain_norm, "route": _plain_route, "adamw": _plain_adamw, "sample": _plain_sample}
        return plain[case["op"]](st)
    g = _g()
    if case["op"] == "norm":
        out, mean, rstd = g.gmm_layer_norm(st["X"], st["gamma"], st["beta"], eps=EPS)
        if not case["grad"]:
            return out, mean, rstd
        return (out, mean, rstd) + tuple(g.gmm_layer_norm_grad(st["dout"], st["X"], mean, rstd, gamma=st["gamma"]))
    if case["op"] == "route":
        how = dict(score=case["score"], renormalize=case["renorm"], scale=2.5)
        idx, weights = g.gmm_route_topm(st["logits"], case["m"], bias=st["bias"], groups=case["groups"],
                                        keep_groups=case["keep"], group_top=case["top"], **how)
        if not case["grad"]:
            return idx, weights
        return idx, weights, g.gmm_route_topm_grad(st["dweights"], st["logits"], idx, dscores=st["dscores"], **how)
    if case["op"] == "adamw":
        scales = dict(m_scale=st["ms"], v_scale=st["vs"]) if case["bits"] == 8 else {}
        g.gmm_adamw_step(st["p"], st["g"], st["m"], st["v"], st["step"], norm=st["norm"],
                         copies=st["copy"] if case["copies"] else None, **scales, **ADAMW)
        st["step"] += 1
        return st["p"], st["m"], st["v"], st["ms"], st["vs"], st["copy"]
    return g.gmm_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                        min_p=st["min_p"])


# ---------------------------------------------------------------- what a pass needs

def work(case):
    if case["op"] == "norm":
        N, D, e = case["N"], case["D"], BYTES[case["dtype"]]
        b, f = e * (2 * N * D + 2 * D) + 8 * N, 8 * N * D
        if case["grad"]:
            b, f = b + 2 * e * N * D + 8 * D, f + 14 * N * D
        return {"bytes": b, "flops": f}
    if case["op"] == "route":
        N, E, m, e = case["N"], case["E"], case["m"], BYTES[case["dtype"]]
        b, f = e * N * E + (4 * E if case["bias"] else 0) + 8 * N * m, 5 * N * E
        if case["grad"]:
            b, f = b + e * N * E + 4 * N * m + 4 * E, f + 5 * N * E
        return {"bytes": b, "flops": f}
    if case["op"] == "adamw":
        b = 0
        for n, (tp, tg) in zip(_sizes(case), _types(case)):
            states = 16 * n if case["bits"] == 32 else 4 * n + 16 * ((n + BLOCK - 1) // BLOCK)
            b += 2 * BYTES[tp] * n + BYTES[tg] * n + states + (2 * n if case["copies"] else 0)
        return {"bytes": b + 4, "flops": 15 * sum(_sizes(case))}
    return {"bytes": BYTES[case["dtype"]] * case["N"] * case["V"] + 12 * case["N"], "flops": 4 * case["N"] * case["V"]}


# ---------------------------------------------------------------- 64 bits

def _exact_norm(st):
    """Through torch's float64 variance; the rows' gradient as the projection of
    q off the rows' mean and normalised direction."""
    X = st["X"].double()
    D = X.shape[1]
    var, mean = torch.var_mean(X, dim=1, correction=0, keepdim=True)
    rstd = (var + EPS).rsqrt()
    y = (X - mean).mul_(rstd)
    out = torch.addcmul(st["beta"].double(), y, st["gamma"].double())
    if not st["case"]["grad"]:
        return out, mean[:, 0], rstd[:, 0]
    dy = st["dout"].double()
    dgamma, dbeta = torch.einsum("nd,nd->d", dy, y), dy.sum(0)
    q = dy * st["gamma"].double()
    dX = (q - q.mean(1, keepdim=True) - y * (torch.einsum("nd,nd->n", q, y) / D)[:, None]) * rstd
    return out, mean[:, 0], rstd[:, 0], dX, dgamma, dbeta


def _exact_route(st):
    """The codes by repeated maxima, the gradient by torch's differentiation."""
    c = st["case"]
    N, E, G = c["N"], c["E"], c["groups"]
    l = st["logits"].double().requires_grad_()  # noqa: E741
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    s = torch.nan_to_num(s, 0.0)  # a row without experts
    with torch.no_grad():
        off = torch.isneginf(l)
        key = (s + st["bias"].double() if st["bias"] is not None else s.clone()).masked_fill(off, -math.inf)
        if G > 1:
            parts = key.unflatten(1, (G, -1))
            top = parts.topk(min(c["top"], E // G), dim=2).values
            score = top.masked_fill(top == -math.inf, 0.0).sum(2).masked_fill(top[:, :, 0] == -math.inf, -math.inf)
            allowed = torch.zeros_like(score, dtype=torch.bool)
            for _ in range(c["keep"]):
                allowed.scatter_(1, score.argmax(1, keepdim=True), True)
                score = score.masked_fill(allowed, -math.inf)
            key = parts.masked_fill(~allowed[:, :, None], -math.inf).flatten(1)
        if st["bias"] is None:
            key = l.detach().masked_fill(key == -math.inf, -math.inf)
        found = []
        for _ in range(c["m"]):
            best = key.max(1, keepdim=True).values
            at = (key == best).to(torch.uint8).argmax(1, keepdim=True)
            found.append(torch.where(best > -math.inf, at, torch.full_like(at, -1)))
            key = key.scatter(1, at, -math.inf)
        idx = torch.cat(found, 1)
    on = (idx >= 0).double()
    w = s.gather(1, idx.clamp(min=0)) * on
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    w = 2.5 * w
    if not c["grad"]:
        return idx.to(torch.int32), w.detach()
    ((w * st["dweights"].double()).sum() + (s * st["dscores"].double()).sum()).backward()
    return idx.to(torch.int32), w.detach(), torch.nan_to_num(l.grad, 0.0)


def _exact_round(x, d, floor):
    """Values of one block's states on the e4m3 grid: the two neighbours, and which of them the number d picks."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    low = torch.floor(a / step) * step
    r = torch.where((a - low) / step + d.double() / 65536.0 >= 1.0, low + step, low).clamp(max=448.0)
    if floor:
        r = torch.where(x > 0.0, r.clamp(min=2.0 ** -9), r)
    return torch.sign(x) * r


def _exact_adamw(st):
    c, o = st["case"], ADAMW
    (b1, b2), t = o["betas"], st["step"]
    scale = min(1.0, o["max_norm"] / (float(st["norm"].double()) + 1e-6))
    out = [[] for _ in range(6)]
    for j in range(c["tensors"]):
        p, g = st["p"][j].double(), st["g"][j].double() * scale
        n = p.numel()
        m, v = st["m"][j].double(), st["v"][j].double()
        if c["bits"] == 8:
            block = torch.arange(n, device="cuda") // BLOCK
            m, v = m * st["ms"][j].double()[block], (v * st["vs"][j].double()[block]) ** 2
        m, v = torch.lerp(g, m, b1), torch.lerp(g * g, v, b2)
        p = p - o["lr"] * (o["weight_decay"] * p + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + o["eps"]))
        out[0].append(p)
        if c["copies"]:
            out[5].append(p)
        if c["bits"] == 32:
            out[1].append(m)
            out[2].append(v)
            continue
        for k, (x, d) in enumerate(zip((m, v.sqrt()), _dither(n, j, t, o["seed"]))):
            top = torch.zeros(block[-1] + 1, device="cuda", dtype=torch.float64).index_reduce_(0, block, x.abs(), "amax")
            out[1 + k].append(_exact_round(x * (448.0 / top)[block], d, k == 1))
            out[3 + k].append(top / 448.0)
    return tuple(out)


def _exact_sample(st):
    """Row by row over the nonzero settings: thresholds from the sorted probabilities, the token by bisection."""
    c = st["case"]
    tokens, logps = [], []
    at = lambda k, r: float(st[k][r]) if isinstance(st[k], torch.Tensor) else st[k]  # noqa: E731
    for r in range(c["N"]):
        l, T = st["logits"][r].double(), at("temperature", r)  # noqa: E741
        if not T > 0:
            tokens.append(int((l == l.max()).nonzero()[0]))
            logps.append(0.0)
            continue
        p = torch.softmax(l / T, 0)
        order = torch.sort(l, descending=True, stable=True).indices
        desc = p[order]
        keep = c["V"]
        k = int(at("top_k", r))
        if 0 < k < keep:
            keep = k
        share = at("top_p", r)
        if share < 1.0:
            total = torch.cumsum(desc[:keep], 0)
            keep = min(keep, 1 + int((total < share * total[-1]).sum()))
        keep = min(keep, max(1, int((desc >= min(at("min_p", r), 1.0) * desc[0]).sum())))
        chosen = order[:keep].sort().values
        mass = torch.cumsum(p[chosen], 0)
        i = min(keep - 1, int(torch.searchsorted(mass, st["u"][r].double() * mass[-1], right=True)))
        tokens.append(int(chosen[i]))
        logps.append(float(torch.log(p[chosen[i]] / mass[-1])))
    return torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.tensor(logps, dtype=torch.float64, device="cuda")


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "adamw": _exact_adamw, "sample": _exact_sample}[case["op"]](st)
