"""Plain 64-bit forms of layer norm, routing, AdamW and sampling, and the error
bounds that their tests allow (u = 2^-24 for a float32 operation, half = eps / 2
for one rounding to the rows' type, as in head_ref)."""
import math

import numpy as np
import torch

from head_ref import U, half, tiny

F32_MAX = float(torch.finfo(torch.float32).max)


def norm(X, gamma=None, beta=None, eps=1e-5):
    """out, mean, rstd in float64 and a bound for each.

    A sum has at most 64 adds in a thread, 6 in a wave and 16 over waves: under
    100.  The first mean is off by 100 u mean|x|, and the differences from it are
    corrected by their own mean, which is off by 100 u of mean|d|, d = x - mean:
      mean: both and one rounding;  d: those and two roundings of its own
      var:  100 u and the differences' roundings, beside the square of what the
            first mean is off by (times the sum's own 100 u) where all x are equal
      out:  the relative errors of d, rstd and two products, one add, one rounding
    """
    x = X.reshape(-1, X.shape[-1]).double()
    g = 1.0 if gamma is None else gamma.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64, device=x.device) if beta is None else beta.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    out = d * rstd * g + b
    first = 100 * U * x.abs().mean(1, keepdim=True)
    e_mean = 100 * U * (d.abs().mean(1, keepdim=True) + first) + first * 4 * U
    e_d = e_mean + 3 * U * (d.abs() + first)
    e_var = 110 * U * (var + first * first) + 2 * e_mean * first + 2 * (d.abs() * e_d).mean(1, keepdim=True)
    e_rstd = rstd * (0.5 * e_var / (var + eps) * 1.01 + 4 * U)
    tol = (e_d * rstd + d.abs() * e_rstd) * (g.abs() if gamma is not None else 1.0) + 4 * U * ((out - b).abs() + b.abs())
    tol = tol + half(X.dtype) * (out.abs() + tol) + tiny(X.dtype)
    lead = X.shape[:-1]
    return ((out.reshape(X.shape), tol.reshape(X.shape)), (mean.reshape(lead), (e_mean + 2 * U * mean.abs()).reshape(lead)),
            (rstd.reshape(lead), e_rstd.reshape(lead)))


def norm_grad(dout, X, mean, rstd, gamma=None, old=None):
    """dX, dgamma, dbeta with bounds, for the float32 mean and rstd of the call.

    xh: three roundings; a sum over a row: 100 adds; over the rows: a thread's
    chain of at most R / 64 and under 100 joins, each term with five roundings.
    old: what accumulate added to (one more add)."""
    x, y = (t.reshape(-1, X.shape[-1]).double() for t in (X, dout))
    R, D = x.shape
    m, r = mean.reshape(-1, 1).double(), rstd.reshape(-1, 1).double()
    g = torch.ones(D, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    xh, q = (x - m) * r, y * g
    a, b = q.mean(1, keepdim=True), (q * xh).mean(1, keepdim=True)
    dX = r * (q - a - xh * b)
    e = (8 * U * (q.abs() + a.abs() + (xh * b).abs()) + 100 * U * q.abs().mean(1, keepdim=True)
         + xh.abs() * 110 * U * (q * xh).abs().mean(1, keepdim=True))
    out = [dX, (y * xh).sum(0), y.sum(0)]
    chain = (R // 64 + 105) * U
    tol = [r.abs() * e + 2 * U * dX.abs(), chain * (y * xh).abs().sum(0), chain * y.abs().sum(0)]
    if old is not None:
        for i, t in enumerate(old):
            out[i] = out[i] + t.double().reshape(out[i].shape)
            tol[i] = tol[i] + 2 * U * (out[i].abs() + tol[i])
    tol[0] = tol[0] + half(X.dtype) * (out[0].abs() + tol[0]) + tiny(X.dtype)
    return (out[0].reshape(X.shape), tol[0].reshape(X.shape)), (out[1], tol[1] + 2 * U * out[1].abs()), \
        (out[2], tol[2] + 2 * U * out[2].abs())


def scores(logits, score):
    """float64 scores of every expert (0 where it is off) and which are on."""
    l = logits.detach().double().cpu().numpy()  # noqa: E741
    on = l > -math.inf  # False for NaN
    l = np.where(on, np.minimum(l, F32_MAX), -math.inf)  # noqa: E741
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return l, np.where(on, 1.0 / (1.0 + np.exp(-np.where(on, l, 0.0))), 0.0), on
        top = np.where(on.any(-1), l.max(-1), 0.0)[..., None]
        e = np.where(on, np.exp(l - top), 0.0)
        return l, e / np.maximum(e.sum(-1, keepdims=True), 1e-300), on


def route(logits, m, bias=None, score="softmax", groups=1, keep=None, top=1, renorm=True, scale=1.0):
    """idx (-1 behind the last) and weights in float64, row by row."""
    l, s, on = scores(logits.reshape(-1, logits.shape[-1]), score)  # noqa: E741
    R, E = l.shape
    b = None if bias is None else bias.double().cpu().numpy()
    keep = groups if keep is None else keep
    idx, w = np.full((R, m), -1, np.int32), np.zeros((R, m))
    for r in range(R):
        t = l[r] if b is None else s[r] + b
        allowed = on[r].copy()
        if groups > 1:
            gt = s[r] if b is None and top == 2 else t
            def value(g):
                best = sorted((gt[e] for e in range(g * (E // groups), (g + 1) * (E // groups)) if on[r, e]), reverse=True)
                return sum(best[:top]) if best else -math.inf
            value = [value(g) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:keep]
            allowed &= np.isin(np.arange(E) // (E // groups), kept)
        order = sorted((e for e in range(E) if allowed[e]), key=lambda e: (-t[e], e))[:m]
        idx[r, :len(order)] = order
        q = s[r, order]
        if renorm and len(order):
            if score == "softmax":  # a sum that does not vanish
                q = np.exp(l[r, order] - l[r, order].max())
            q = q / max(q.sum(), 1e-300)
        w[r, :len(order)] = scale * q
    lead = tuple(logits.shape[:-1]) + (m,)
    return torch.from_numpy(idx.reshape(lead)), torch.from_numpy(w.reshape(lead))


def route_grad(dweights, logits, idx, score="softmax", renorm=True, scale=1.0, dscores=None):
    """dlogits in float64 and its bound.

    A score: exp of a rounded difference (u |l - max l| relative, at most 128: below
    exp(-128) of the row it is nothing), 2 ulp of exp, a sum and a quotient; every
    product and sum behind it a rounding, under 64 in all, over the absolute sum
    of what is added."""
    l, s, on = (torch.from_numpy(a) for a in scores(logits.reshape(-1, logits.shape[-1]), score))  # noqa: E741
    R, E = s.shape
    m = idx.shape[-1]
    idx2 = idx.reshape(R, m).cpu().long()
    live = torch.cumprod(((idx2 >= 0) & (idx2 < E)).long(), 1).bool()
    at = torch.where(live, idx2, torch.zeros_like(idx2))
    dw = torch.zeros(R, m, dtype=torch.float64) if dweights is None else dweights.reshape(R, m).double().cpu()
    u = torch.where(live, scale * dw, torch.zeros_like(dw))
    rest = torch.ones_like(s) if score == "softmax" else 1.0 / (1.0 + torch.exp(torch.where(on, l, torch.zeros_like(l))))
    ds = torch.zeros(E, dtype=torch.float64) if dscores is None else dscores.double().cpu()
    ds = ds.expand(R, E).clone()
    ads = ds.abs()
    direct, adirect = torch.zeros_like(s), torch.zeros_like(s)
    if renorm:
        sel = torch.where(live, l.gather(1, at), torch.full_like(u, -math.inf))
        if score == "softmax":
            q = torch.exp(sel - sel.max(1, keepdim=True).values.clamp_min(-F32_MAX))
        else:
            q = torch.where(live, s.gather(1, at), torch.zeros_like(u))
        q = torch.where(live, q / q.sum(1, keepdim=True).clamp_min(1e-300), torch.zeros_like(u))
        mean, amean = (q * u).sum(1, keepdim=True), (q * u.abs()).sum(1, keepdim=True)
        direct.scatter_add_(1, at, q * (u - mean) * live)
        adirect.scatter_add_(1, at, q * (u.abs() + amean) * live)
    else:
        ds.scatter_add_(1, at, u)
        ads.scatter_add_(1, at, u.abs())
    c, ac = torch.zeros(R, 1, dtype=torch.float64), torch.zeros(R, 1, dtype=torch.float64)
    if score == "softmax":
        c, ac = (ds * s).sum(1, keepdim=True), (ads * s).sum(1, keepdim=True)
    out = torch.where(on, direct * rest + s * rest * (ds - c), torch.zeros_like(s))
    mag = adirect * rest + s * rest * (ads + ac)
    spread = torch.where(on, (l.max(1, keepdim=True).values - l).clamp(0, 128), torch.zeros_like(l)).max()
    tol = torch.where(on, U * (2 * spread + 64) * mag + 2.0 ** -149 * 64, torch.zeros_like(mag))
    tol = tol + half(logits.dtype) * (out.abs() + tol) + tiny(logits.dtype)
    return out.reshape(logits.shape), tol.reshape(logits.shape)


# ---------------------------------------------------------------- AdamW

def mix(x):
    x = ((x ^ (x >> np.uint32(16))) * np.uint32(0x9E3779B1)).astype(np.uint32)
    x = ((x ^ (x >> np.uint32(15))) * np.uint32(0x6A09E667)).astype(np.uint32)
    return x ^ (x >> np.uint32(16))


def dither(n, tensor, step, seed):
    """The 16-bit numbers of the first and of the second moments."""
    with np.errstate(over="ignore"):
        u = np.uint32
        key = mix(mix(np.array([(seed + 0x9E3779B1 * step) & 0xFFFFFFFF], u)) ^ u(tensor))
        i = np.arange(n, dtype=np.uint64)
        h = mix((mix(key + (i // 256).astype(u)) + (i % 256).astype(u) * u(0x9E3779B1)).astype(u))
    return h >> u(16), h & u(0xffff)


def encode(x, d, root):
    """float32 x to (e4m3 bytes, scales), every operation in float32."""
    f = np.float32
    n = len(x)
    pad = np.concatenate([x, np.zeros(-n % 256, f)]).reshape(-1, 256)
    top = np.abs(pad).max(1)
    none = top < f(2.0 ** -100)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        s = np.where(none, f(0), top * (f(1) / f(448))).astype(f)
        inv = np.where(none, f(0), f(1) / top * f(448)).astype(f)
        y = (pad * inv[:, None]).reshape(-1)[:n].astype(f)
    a = np.minimum(np.abs(y), f(448)).astype(f)
    up = ((a.view(np.uint32) + (d << np.uint32(4))) >> np.uint32(20)).astype(np.int64) - (120 << 3)
    low = (a * f(512) + d.astype(f) * f(2.0 ** -16)).astype(f).astype(np.int64)
    c = np.where(a < f(2.0 ** -6), low, up)
    if root:
        c = np.where((y > 0) & (c == 0), 1, c)
    else:
        c = np.where((y < 0) & (c != 0), c | 0x80, c)
    return np.where(np.isnan(y), 0x7f, c).astype(np.uint8), s


def decode(c, s):
    """e4m3 bytes and scales to float32 values."""
    mag = c & 0x7f
    bits = (mag.astype(np.uint32) << np.uint32(20)) + np.uint32(120 << 23)
    v = np.where(mag < 8, mag.astype(np.float32) * np.float32(2.0 ** -9), bits.view(np.float32))
    v = np.where(mag == 0x7f, np.float32(np.nan), np.where(c & 0x80, -v, v)).astype(np.float32)
    return (v * np.repeat(s, 256)[:len(c)]).astype(np.float32)


def adamw(p, g, m, v, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, clip=1.0, real=np.float32):
    """One step on float32 arrays in the library's order of operations; real =
    np.float64: the formula itself.  Returns p, m, v, sqrt(v)."""
    f = real
    g = (f(np.float32(clip) if f is np.float32 else clip) * g.astype(f)).astype(f)
    b1, b2 = betas
    with np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore"):
        m = (f(b1) * m.astype(f) + f(1.0 - b1) * g).astype(f)
        v = (f(b2) * v.astype(f) + f(1.0 - b2) * (g * g)).astype(f)
        alpha = f(lr / -math.expm1(step * math.log(b1)) if b1 else lr)
        root = f(1.0 / math.sqrt(-math.expm1(step * math.log(b2))) if b2 else 1.0)
        r = np.sqrt(v).astype(f)
        p = (p.astype(f) * f(1.0 - lr * weight_decay) - alpha * (m / (r * root + f(eps)))).astype(f)
    return p, m, v, r


# ---------------------------------------------------------------- sampling

def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log of its share, how sure) of one float64 row of logits: weights as
    integers of S bits, sums exact.  `sure` is False where a threshold lies nearer
    to a sum than the float64 exponential's own error (2 ulp a weight) may move it."""
    V = len(row)
    S = min(52, 62 - max(0, (V - 1).bit_length()))
    on = [i for i in range(V) if row[i] > -math.inf]
    if not on:
        return -1, -math.inf, True
    x = np.minimum(row, F32_MAX)
    order = sorted(on, key=lambda i: (-x[i], i))
    if not temperature > 0:
        return order[0], 0.0, True
    with np.errstate(over="ignore"):
        z = (x - x[order[0]]) / temperature
    e = {i: math.exp(z[i]) for i in order}
    w = {i: round(e[i] * 2.0 ** S) for i in order}
    off = {i: 0 if e[i] in (0.0, 1.0) else 1 + int(w[i] * 2.0 ** -51) for i in order}  # what w may be off by
    sure = True
    kept = order[:top_k] if top_k > 0 else order
    if top_p < 1.0:
        target, before, slack = top_p * float(sum(w[i] for i in kept)), 0, top_p * sum(off[i] for i in kept)
        n = 0
        for i in kept:
            if n and not float(before) < target:
                break
            before += w[i]
            slack += off[i]
            sure &= slack == 0 or abs(before - target) > slack
            n += 1
        kept = kept[:n]
    least = min(min_p, 1.0)
    if least > 0:
        sure &= all(off[i] == 0 or abs(e[i] - least) > 1e-14 for i in kept)
        kept = [i for i in kept if e[i] >= least]
    kept = sorted(kept)
    total, slack = sum(w[i] for i in kept), sum(off[i] for i in kept)
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    target, run = u * float(total), 0
    found = None
    for i in kept:
        run += w[i]
        sure &= slack == 0 or u == 0.0 or abs(run - target) > 2 * slack + 2.0 ** -52 * total
        if found is None and float(run) > target:
            found = i
    return found, z[found] - math.log(total * 2.0 ** -S), sure
