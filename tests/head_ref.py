"""Plain 64-bit forms of the softmax head, codebook and clipping operators, and
the error bounds that their tests allow.

Bounds are elementwise and follow from the arithmetic: u = 2^-24 for a float32
operation, half = eps / 2 for one rounding to the rows' type.
"""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the smallest values of a type (subnormals)."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def xent(X, W, labels, bias=None, gloss=None, rows=1 << 13):
    """loss, lse, dX, dW, db in float64 and a bound for each.

    l:    a product of D terms summed in float32, any order, and the bias:
          E_l <= (D + 4) u (sum_d |x_d w_vd| + |b_v|); E is its maximum over v
    lse:  E, then the exponentials and their sum: 256 u covers the argument's
          rounding over the spread that carries weight and the longest chain
          of adds (16 in a lane, 6 in a wave, under 200 over tiles), 4 u |lse|
          the subtraction and the final add
    loss: both and one subtraction
    G:    |g| p (E + E_lse + 16 u) + 8 u |G|, rounded once to the rows' type
          after a scaling (two more roundings of 32 bits; half rows: to 2^15 max
          |g|, so that what vanishes is below 2^-39 max |g|)
    dX:   sum_v dG |w| + V u sum |G| |w|, rounded once; dW, db likewise
    """
    X2 = X.reshape(-1, X.shape[-1]).double()
    W2, y = W.double(), labels.reshape(-1).long()
    R, D = X2.shape
    V = W2.shape[0]
    dt = X.dtype
    h = half(dt) if dt != torch.float32 else 0.0
    b = torch.zeros(V, dtype=torch.float64, device=X.device) if bias is None else bias.double()
    g = torch.ones(R, dtype=torch.float64, device=X.device) if gloss is None else gloss.reshape(-1).double()
    live = y >= 0
    g = torch.where(live, g, torch.zeros_like(g))
    gmax = float(g.abs().max()) if R else 0.0
    out = {k: torch.zeros(s, dtype=torch.float64, device=X.device)
           for k, s in (("loss", R), ("lse", R), ("dX", (R, D)), ("dW", (V, D)), ("db", V))}
    tol = {k: torch.zeros_like(v) for k, v in out.items()}
    finite_b = torch.where(torch.isfinite(b), b, torch.zeros_like(b))
    for r0 in range(0, R, rows):
        s = slice(r0, min(R, r0 + rows))
        x = torch.where(live[s, None], X2[s], torch.nan_to_num(X2[s], 0.0, 0.0, 0.0))
        L = x @ W2.t() + b
        E = ((D + 4) * U * (x.abs() @ W2.abs().t() + finite_b.abs())).max(dim=1).values
        z = torch.logsumexp(L, dim=1)
        e_z = E + U * (256 + 4 * z.abs())
        at = y[s].clamp_min(0)
        ly = L.gather(1, at[:, None])[:, 0]
        out["lse"][s], tol["lse"][s] = z, e_z
        out["loss"][s] = torch.where(live[s], z - ly, torch.zeros_like(z))
        tol["loss"][s] = torch.where(live[s], E + e_z + 2 * U * (z - ly).abs(), torch.zeros_like(z))
        P = torch.exp(L - z[:, None])
        G = P.clone()
        G[torch.arange(len(at), device=X.device), at] -= 1.0
        G = torch.where(live[s, None], G * g[s, None], torch.zeros_like(G))
        dG = g[s, None].abs() * P * (E + e_z + 16 * U)[:, None] + 8 * U * G.abs()
        one_minus = g[s].abs() * (E + e_z + 16 * U)  # p - 1 keeps p's absolute error, p <= 1
        dG.scatter_add_(1, at[:, None], (one_minus * 4)[:, None])
        dG = torch.where(live[s, None], dG, torch.zeros_like(dG))
        dGr = dG + h * (G.abs() + dG) + (2.0 ** -39 * gmax if dt == torch.float16 else 0.0) * (h > 0)
        dGr = torch.where(live[s, None], dGr, torch.zeros_like(dGr))
        out["dX"][s] = G @ W2
        tol["dX"][s] = dGr @ W2.abs() + (V + 8) * U * (G.abs() @ W2.abs())
        out["dW"] += G.t() @ x
        tol["dW"] += dGr.t() @ x.abs() + (R + 8) * U * (G.abs().t() @ x.abs())
        out["db"] += G.sum(0)
        tol["db"] += dG.sum(0) + (R + 8) * U * G.abs().sum(0)
    for k in ("dX", "dW"):
        tol[k] += (half(dt) + 2 * U) * (out[k].abs() + tol[k]) + tiny(dt)
    tol["db"] += 2 * U * out["db"].abs()
    shape = {"loss": labels.shape, "lse": labels.shape, "dX": X.shape}
    for d in (out, tol):
        for k, v in shape.items():
            d[k] = d[k].reshape(v)
    return out, tol


def entries(idx, K):
    """Which slots of idx (.., m) hold codes: the leading values in [0, K)."""
    ok = (idx >= 0) & (idx < K)
    return torch.cumprod(ok.long(), dim=-1).bool()


def lookup(table, idx, weights=None, scale=1.0):
    """Rows rebuilt from codes, with table (K, D) and idx (N, m): float64 and bound.
    m products and adds in float32, the scale, one rounding."""
    live = entries(idx, table.shape[0])
    w = live.double() if weights is None else torch.where(live, weights.double(), torch.zeros(1, dtype=torch.float64, device=idx.device))
    rows = table.double()[torch.where(live, idx, torch.zeros_like(idx)).long()]
    out = scale * (w[..., None] * rows).sum(dim=-2)
    mag = abs(scale) * (w.abs()[..., None] * rows.abs()).sum(dim=-2)
    tol = (idx.shape[-1] + 2) * U * mag
    return out, tol + half(table.dtype) * (out.abs() + tol) + tiny(table.dtype)


def lookup_grad(dout, idx, K, table=None, weights=None, scale=1.0, old=None):
    """dtable, dweights with bounds: a code's n entries are n float32 products and adds."""
    live = entries(idx, K)
    N, m = idx.shape
    D = dout.shape[-1]
    w = live.double() if weights is None else torch.where(live, weights.double(), torch.zeros(1, dtype=torch.float64, device=idx.device))
    row = torch.arange(N, device=idx.device)[:, None].expand(N, m)[live]
    code, we = idx[live].long(), w[live]
    d = dout.double()
    res = torch.zeros(K, D, dtype=torch.float64, device=idx.device)
    mag = torch.zeros_like(res)
    res.index_add_(0, code, scale * we[:, None] * d[row])
    mag.index_add_(0, code, (abs(scale) * we.abs())[:, None] * d[row].abs())
    n = torch.bincount(code, minlength=K).double()[:, None]
    tol = (n + 4) * U * mag
    if old is not None:
        res = res + old.double()
        tol = tol + 2 * U * (res.abs() + old.double().abs())
    tol = tol + half(dout.dtype) * (res.abs() + tol) + tiny(dout.dtype)
    if table is None:
        return (res, tol), None
    t = table.double()[torch.where(live, idx, torch.zeros_like(idx)).long()]
    dw = scale * (d[:, None, :] * t).sum(-1) * live
    dmag = abs(scale) * (d.abs()[:, None, :] * t.abs()).sum(-1) * live
    return (res, tol), (dw, (D + 8) * U * dmag)


def within(name, got, want, tol):
    """Every element inside its bound; NaN only where NaN is wanted."""
    got = got.double()
    want, tol = want.reshape(got.shape), tol.reshape(got.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaN where there should be none, or none where there should be"
    err = torch.where(nan | (got == want), torch.zeros_like(got), (got - want).abs())
    over = err > tol
    if over.any():
        i = int((err / tol.clamp_min(1e-300)).argmax())
        raise AssertionError(f"{name}: {int(over.sum())} of {over.numel()} values outside their bound; worst at flat "
                             f"index {i}: got {got.flatten()[i].item()!r}, want {want.flatten()[i].item()!r}, "
                             f"bound {tol.flatten()[i].item():.3e}")
