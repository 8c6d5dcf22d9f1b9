"""Refusals of the layer norm, routing, AdamW and sampling calls that need no
GPU: the arguments are validated on the host before any device work."""
import ctypes
import math

import pytest

from soft_clustering_em_amd import _abi

P = ctypes.c_void_p
A, B, C, E, F, G_, H = (P(i << 40) for i in range(1, 8))
WS, BIG = P(1 << 50), 1 << 60
INV, UNS, WSE = _abi.GMM_ERR_INVALID_ARG, _abi.GMM_ERR_UNSUPPORTED, _abi.GMM_ERR_WORKSPACE


def rows(N=100, D=64, Bn=1, dtype=_abi.DT_BF16, ld=None, x=A, sb=None):
    ld = D if ld is None else ld
    return _abi.GmmData(x, dtype, Bn, N, D, ld, N * ld if sb is None else sb)


def last():
    return _abi.lib().gmm_last_error().decode()


BAD_ROWS = [(dict(D=0, ld=0), INV), (dict(N=-1), INV), (dict(Bn=0), INV), (dict(ld=63), INV), (dict(Bn=2, sb=100), INV),
            (dict(x=None), INV), (dict(dtype=7), INV), (dict(N=1 << 31), UNS), (dict(N=1 << 20, Bn=1 << 11), UNS),
            (dict(x=P((1 << 40) + 1)), INV)]


def norm(r=None, gamma=B, beta=C, dt=_abi.DT_BF16, eps=1e-5, out=E, mean=F, rstd=G_):
    return _abi.lib().gmm_layer_norm(ctypes.byref(rows(**(r or {}))), gamma, beta, dt, eps, out, mean, rstd, None)


def norm_grad(r=None, d=None, mean=C, rstd=E, gamma=F, dt=_abi.DT_BF16, dx=G_, dg=H, db=P(8 << 40), ws=WS, have=BIG):
    y = rows(**{**dict(x=B), **(r or {}), **(d or {})})
    return _abi.lib().gmm_layer_norm_grad(ctypes.byref(y), ctypes.byref(rows(**(r or {}))), mean, rstd, gamma, dt, dx, dg, db, 0,
                                          ws, have, None)


@pytest.mark.parametrize("r,status", BAD_ROWS + [(dict(D=32769), UNS)])
def test_norm_refuses_bad_rows(r, status):
    assert norm(r) == status and last()
    assert norm_grad(r, d=dict(x=B)) == status and last()
    assert _abi.lib().gmm_layer_norm_grad_workspace_bytes(ctypes.byref(rows(**r)), 7) == 0


def test_norm_refusals():
    for kw in (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(out=None), dict(dt=5), dict(gamma=P((2 << 40) + 1)),
               dict(out=P((5 << 40) + 1)), dict(mean=P((6 << 40) + 2)), dict(out=A), dict(out=P((1 << 40) + 100)), dict(out=B),
               dict(mean=C), dict(mean=G_), dict(rstd=E)):
        assert norm(**kw) == INV and last(), kw
    assert norm(dt=_abi.DT_F16) == UNS
    assert "overlaps" in (norm(out=A), last())[1]


def test_norm_grad_refusals():
    for kw in (dict(mean=None), dict(rstd=None), dict(dx=None, dg=None, db=None), dict(d=dict(N=99)), dict(d=dict(D=32, ld=32)),
               dict(dx=A), dict(dx=B), dict(dx=C), dict(dg=F), dict(dg=G_), dict(db=H), dict(dx=P((7 << 40) + 1)), dict(dg=P((7 << 40) + 2))):
        assert norm_grad(**kw) == INV and last(), kw
    assert norm_grad(d=dict(dtype=_abi.DT_F32)) == UNS and norm_grad(dt=_abi.DT_F16) == UNS
    n = _abi.lib().gmm_layer_norm_grad_workspace_bytes(ctypes.byref(rows()), 7)
    assert n % 256 == 0 and n > _abi.lib().gmm_layer_norm_grad_workspace_bytes(ctypes.byref(rows()), 1) > 0
    for ws, have in ((None, BIG), (P((1 << 50) + 8), BIG), (WS, n - 1)):
        assert norm_grad(ws=ws, have=have) == WSE
    f = lambda N, D: _abi.lib().gmm_layer_norm_grad_workspace_bytes(ctypes.byref(rows(N=N, D=D)), 7)  # noqa: E731
    assert f(1 << 20, 2048) == f(1 << 24, 2048) <= 1 << 25 and f(1 << 20, 32768) <= 1 << 25


def how(score=0, groups=1, keep=1, top=1, renorm=1, scale=1.0):
    return _abi.GmmRouting(score, groups, keep, top, renorm, scale)


def route(r=None, h=None, m=4, bias=B, idx=C, w=E):
    return _abi.lib().gmm_route_topm(ctypes.byref(rows(**(r or {}))), bias, ctypes.byref(how(**(h or {}))), m, idx, w, None)


def route_grad(r=None, h=None, m=4, idx=B, dw=C, ds=E, dl=F):
    return _abi.lib().gmm_route_topm_grad(ctypes.byref(rows(**(r or {}))), ctypes.byref(how(**(h or {}))), m, idx, dw, ds, dl, None)


@pytest.mark.parametrize("r,h,m,status", [(r, {}, 4, s) for r, s in BAD_ROWS] + [
    (dict(D=1025), {}, 4, UNS), ({}, dict(score=2), 4, INV), ({}, {}, 0, INV), ({}, {}, 17, INV), ({}, dict(groups=0), 4, INV),
    ({}, dict(groups=3), 4, INV), (dict(D=130), dict(groups=65), 4, UNS), ({}, dict(groups=4, keep=5), 4, INV),
    ({}, dict(groups=4, keep=0), 4, INV), ({}, dict(top=3), 4, INV), ({}, dict(top=0), 4, INV), ({}, dict(scale=math.nan), 4, INV)])
def test_route_refuses_bad_operands(r, h, m, status):
    assert route(r, h, m) == status and last()
    assert route_grad(r, h, m) == status and last()


def test_route_refuses_bad_pointers():
    for kw in (dict(idx=None), dict(w=None), dict(idx=A), dict(w=B), dict(w=C), dict(idx=P((3 << 40) + 2)), dict(bias=P((2 << 40) + 1))):
        assert route(**kw) == INV and last(), kw
    for kw in (dict(idx=None), dict(dw=None, ds=None), dict(dl=None), dict(dl=A), dict(dl=B), dict(dl=C), dict(dl=E),
               dict(dl=P((6 << 40) + 1))):
        assert route_grad(**kw) == INV and last(), kw
    L = _abi.lib()
    assert L.gmm_route_topm(ctypes.byref(rows()), B, None, 4, C, E, None) == INV
    assert L.gmm_route_topm(None, B, ctypes.byref(how()), 4, C, E, None) == INV


def tensor(i, n=100, dtype=0, grad_dtype=0, **kw):
    at = lambda k: ((i * 8 + k + 1) << 40)  # noqa: E731
    a = dict(param=at(0), grad=at(1), m=at(2), v=at(3), m_scale=None, v_scale=None, copy=None, n=n, weight_decay=0.1, dtype=dtype,
             grad_dtype=grad_dtype, copy_dtype=0, reserved=0)
    a.update(kw)
    return _abi.GmmAdamwTensor(**a)


def adamw(ts, count=None, **kw):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, max_norm=1.0, norm=None, step=1, step_dev=None, lr_dev=None, seed=0)
    o.update(kw)
    arr = (_abi.GmmAdamwTensor * max(1, len(ts)))(*ts)
    return _abi.lib().gmm_adamw_step(arr, len(ts) if count is None else count, ctypes.byref(_abi.GmmAdamwOptions(**o)), None)


def test_adamw_refusals():
    ok = [tensor(0), tensor(1, n=300, m_scale=1 << 50, v_scale=1 << 51)]
    for kw in (dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
               dict(eps=-1.0), dict(eps=math.nan), dict(step=0), dict(norm=1 << 52, max_norm=-1.0), dict(norm=1 << 52, max_norm=math.nan),
               dict(norm=(1 << 52) + 2), dict(step_dev=(1 << 52) + 4), dict(lr_dev=(1 << 52) + 1), dict(count=0)):
        assert adamw(ok, **kw) == INV and last(), kw
    for bad in (tensor(2, dtype=3), tensor(2, grad_dtype=-1), tensor(2, copy=1 << 55, copy_dtype=9), tensor(2, n=-1),
                tensor(2, weight_decay=-0.1), tensor(2, weight_decay=math.nan), tensor(2, param=None), tensor(2, m=None), tensor(2, v=None),
                tensor(2, grad=None), tensor(2, m_scale=1 << 55), tensor(2, v_scale=1 << 55), tensor(2, reserved=1),
                tensor(2, param=(17 << 40) + 2), tensor(2, m=(19 << 40) + 1), tensor(2, copy=(1 << 55) + 1, copy_dtype=1)):
        assert adamw(ok + [bad]) == INV and last()
    assert adamw([tensor(0, n=1 << 40)]) == UNS
    assert _abi.lib().gmm_adamw_step(None, 1, ctypes.byref(_abi.GmmAdamwOptions()), None) == INV
    assert _abi.lib().gmm_adamw_step((_abi.GmmAdamwTensor * 1)(tensor(0)), 1, None, None) == INV


def test_adamw_refuses_overlaps():
    p = 1 << 40
    for ts in ([tensor(0, grad=p)], [tensor(0, grad=p + 396)], [tensor(0, m=p)], [tensor(0, v=(3 << 40) + 40)], [tensor(0), tensor(1, param=p)],
               [tensor(0), tensor(1, grad=p + 4)], [tensor(0, copy=2 << 40)], [tensor(0, m_scale=1 << 50, v_scale=1 << 50)],
               [tensor(0, n=300, m_scale=1 << 50, v_scale=(1 << 50) + 4)]):
        assert adamw(ts) == INV and "overlaps" in last()
    for kw in (dict(norm=p + 4), dict(step_dev=(3 << 40) + 8), dict(lr_dev=(4 << 40) + 396)):
        assert adamw([tensor(0)], **kw) == INV and "overlaps" in last()


def sample(r=None, u=B, tokens=C, logp=E, ws=WS, have=BIG, **kw):
    h = dict(temperature=1.0, top_p=0.9, min_p=0.1, top_k=5)
    h.update(kw)
    return _abi.lib().gmm_sample(ctypes.byref(rows(**(r or {}))), ctypes.byref(_abi.GmmSampling(**h)), u, tokens, logp, ws, have, None)


@pytest.mark.parametrize("r,status", BAD_ROWS + [(dict(D=(1 << 24) + 1), UNS)])
def test_sample_refuses_bad_rows(r, status):
    assert sample(r) == status and last()
    assert _abi.lib().gmm_sample_workspace_bytes(ctypes.byref(rows(**r))) == 0


def test_sample_refusals():
    for kw in (dict(u=None), dict(tokens=None), dict(tokens=A), dict(tokens=B), dict(logp=C), dict(logp=P((3 << 40) + 4)), dict(u=P((2 << 40) + 1)),
               dict(temperature=-0.5), dict(temperature=math.nan), dict(top_p=math.nan), dict(min_p=math.nan),
               dict(row_top_k=(1 << 52) + 1), dict(row_top_p=3 << 40), dict(row_temperature=4 << 40)):
        assert sample(**kw) == INV and last(), kw
    n = _abi.lib().gmm_sample_workspace_bytes(ctypes.byref(rows()))
    assert n > 0 and n % 256 == 0
    for ws, have in ((None, BIG), (P((1 << 50) + 16), BIG), (WS, n - 1)):
        assert sample(ws=ws, have=have) == WSE
    assert _abi.lib().gmm_sample(ctypes.byref(rows()), None, B, C, E, WS, BIG, None) == INV


def test_struct_layouts():
    assert ctypes.sizeof(_abi.GmmRouting) == 24 and ctypes.sizeof(_abi.GmmAdamwTensor) == 11 * 8
    assert ctypes.sizeof(_abi.GmmAdamwOptions) == 10 * 8 and ctypes.sizeof(_abi.GmmSampling) == 8 * 8


def test_python_checks_on_the_host():
    """The binding's own checks, with CPU tensors: shapes and types first, then the device."""
    import torch

    import soft_clustering_em_amd as g
    X, v, z = torch.randn(4, 8), torch.ones(8), torch.zeros(4)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    st, st8 = g.new_adamw_state([X]), g.new_adamw_state([X], 8)
    assert st8["m"][0].dtype == torch.float8_e4m3fn and st8["v_scale"][0].shape == (1,)
    step = lambda **kw: g.gmm_adamw_step(**{**dict(params=[X], grads=[X.clone()], step=1, **st), **kw})  # noqa: E731
    for bad in (lambda: g.gmm_layer_norm(X, v[:7]), lambda: g.gmm_layer_norm(X, v, v.half()), lambda: g.gmm_layer_norm(X, v.half()),
                lambda: g.gmm_layer_norm(X.double()), lambda: g.gmm_layer_norm(X.t()), lambda: g.gmm_layer_norm(X),
                lambda: g.gmm_layer_norm_grad(X[:3], X, z, z), lambda: g.gmm_layer_norm_grad(X, X, z[:3], z),
                lambda: g.gmm_layer_norm_grad(X.half(), X, z, z), lambda: g.gmm_layer_norm_grad(X, X, z, z, accumulate=True),
                lambda: g.gmm_layer_norm_grad(X, X, z, z, ws=torch.zeros(1, dtype=torch.uint8).expand(1 << 20)),
                lambda: g.gmm_route_topm(X, 2, score="max"), lambda: g.gmm_route_topm(X, 0), lambda: g.gmm_route_topm(X, 2, bias=v[:5]),
                lambda: g.gmm_route_topm(X, 2, idx=idx.long()), lambda: g.gmm_route_topm(X, 2),
                lambda: g.gmm_route_topm_grad(None, X, idx), lambda: g.gmm_route_topm_grad(z, X, idx),
                lambda: g.gmm_route_topm_grad(torch.zeros(4, 2), X, idx[:3]), lambda: g.gmm_route_topm_grad(None, X, idx, dscores=z),
                lambda: g.new_adamw_state([X], 16), lambda: step(params=[], grads=[]), lambda: step(grads=[X[:3]]),
                lambda: step(params=[X.t()]), lambda: step(params=[X.double()]), lambda: step(m=[X.half()]), lambda: step(norm=z[:1]),
                lambda: step(max_norm=1.0), lambda: step(norm=1.0, max_norm=1.0), lambda: step(copies=[v]), lambda: step(copies=[X.int()]),
                lambda: step(m_scale=[z]), lambda: step(weight_decay=[0.1, 0.2]), lambda: step(step=torch.ones(2, dtype=torch.int64)),
                lambda: step(lr=torch.ones(1, dtype=torch.float64)), lambda: step(**{**st8, "m_scale": [z], "v_scale": [z]}), step,
                lambda: g.gmm_sample(X, z[:3]), lambda: g.gmm_sample(X, z, top_k=z), lambda: g.gmm_sample(X, z, temperature=z.double()),
                lambda: g.gmm_sample(X, z, top_p=z[:2]), lambda: g.gmm_sample(X, z.double()), lambda: g.gmm_sample(X, z)):
        with pytest.raises(ValueError):
            bad()


def test_oracle_encoding_is_e4m3():
    """The oracle's bytes against torch's own e4m3 values, and its roundings to both sides."""
    import numpy as np
    import torch

    import step_ref as ref
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ref.decode(c, np.ones(1, np.float32)), want)
    x = np.concatenate([[np.float32(448)], np.random.default_rng(0).normal(size=255).astype(np.float32) * 10])
    for d in (0, 0xffff):
        b, s = ref.encode(x, np.full(256, d, np.uint32), False)
        v = ref.decode(b, s)
        assert s[0] == 1.0
        grid = np.sort(want[~np.isnan(want)])
        low = np.array([grid[grid <= abs(t)].max() for t in x])
        assert (np.abs(v) >= low).all() and (np.abs(v) - np.abs(x) < np.maximum(np.abs(x) / 8, 2.0 ** -9)).all()
        if d == 0:
            np.testing.assert_array_equal(np.abs(v), low)


def test_dither_is_uniform():
    import numpy as np

    import step_ref as ref
    m, v = ref.dither(1 << 18, 3, 17, 5)
    for d in (m, v):
        counts = np.bincount(d >> 10, minlength=64)
        assert abs(counts - 4096).max() < 6 * 64
        assert abs(np.corrcoef(d[1:], d[:-1])[0, 1]) < 6 / 512 and abs(np.corrcoef(d[256:], d[:-256])[0, 1]) < 6 / 512
    assert abs(np.corrcoef(m, v)[0, 1]) < 6 / 512
    for other in (ref.dither(1 << 18, 3, 18, 5), ref.dither(1 << 18, 4, 17, 5), ref.dither(1 << 18, 3, 17, 6)):
        assert abs(np.corrcoef(m, other[0])[0, 1]) < 6 / 512
