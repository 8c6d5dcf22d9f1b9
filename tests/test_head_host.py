"""Refusals of the softmax head, codebook and clipping calls that need no GPU:
the arguments are validated on the host before any device work."""
import ctypes

import pytest

from soft_clustering_em_amd import _abi

P = ctypes.c_void_p
A, B, C, E, F, G_, H = (P(i << 40) for i in range(1, 8))
WS, BIG = P(1 << 50), 1 << 60


def rows(N=100, D=64, Bn=1, dtype=_abi.DT_BF16, ld=None, x=A, sb=None):
    ld = D if ld is None else ld
    return _abi.GmmData(x, dtype, Bn, N, D, ld, N * ld if sb is None else sb)


def head(V=50, D=64, dtype=_abi.DT_BF16, ld=None, w=B, bias=None):
    return _abi.GmmHead(w, dtype, V, D if ld is None else ld, bias)


def last():
    return _abi.lib().gmm_last_error().decode()


INV, UNS, WSE = _abi.GMM_ERR_INVALID_ARG, _abi.GMM_ERR_UNSUPPORTED, _abi.GMM_ERR_WORKSPACE

BAD_OPERANDS = [
    (dict(D=0, ld=0), {}, INV), (dict(N=-1), {}, INV), (dict(Bn=0), {}, INV), (dict(ld=63), {}, INV),
    (dict(Bn=2, sb=100), {}, INV), (dict(x=None), {}, INV), (dict(dtype=7), {}, INV),
    ({}, dict(V=0), INV), ({}, dict(w=None), INV), ({}, dict(ld=63), INV), ({}, dict(dtype=9), INV),
    ({}, dict(dtype=_abi.DT_F32), UNS), (dict(D=65537), dict(D=65537), UNS), ({}, dict(V=1 << 27), UNS),
    (dict(N=1 << 28), {}, UNS), (dict(N=1 << 18, Bn=1 << 12), {}, UNS), (dict(x=P((1 << 40) + 1)), {}, INV),
    ({}, dict(w=P((2 << 40) + 1)), INV),
]


@pytest.mark.parametrize("r,h,status", BAD_OPERANDS)
def test_xent_refuses_bad_operands(r, h, status):
    L = _abi.lib()
    d, hd = ctypes.byref(rows(**r)), ctypes.byref(head(**h))
    assert L.gmm_softmax_xent(d, hd, C, E, F, WS, BIG, None) == status and last()
    assert L.gmm_softmax_xent_grad(d, hd, C, E, None, F, G_, None, 0, WS, BIG, None) == status and last()
    assert L.gmm_softmax_xent_workspace_bytes(d, hd) == 0
    assert L.gmm_softmax_xent_grad_workspace_bytes(d, hd, 7) == 0


def test_xent_refuses_bad_pointers_and_workspaces():
    L = _abi.lib()
    d, h = ctypes.byref(rows()), ctypes.byref(head())
    assert L.gmm_softmax_xent(None, h, C, E, F, WS, BIG, None) == INV
    assert L.gmm_softmax_xent(d, None, C, E, F, WS, BIG, None) == INV
    for miss in range(3):
        a = [C, E, F]
        a[miss] = None
        assert L.gmm_softmax_xent(d, h, *a, WS, BIG, None) == INV
    assert L.gmm_softmax_xent(d, h, C, E, P((4 << 40) + 8), WS, BIG, None) == INV  # lse inside loss
    for on in (A, B, C):  # loss on the rows, the head, the labels
        assert L.gmm_softmax_xent(d, h, C, on, F, WS, BIG, None) == INV and "overlaps" in last()
    n = L.gmm_softmax_xent_workspace_bytes(d, h)
    assert n > 0 and n % 256 == 0
    for ws, have in ((None, BIG), (P((1 << 50) + 16), BIG), (WS, n - 1)):
        assert L.gmm_softmax_xent(d, h, C, E, F, ws, have, None) == WSE
    n = L.gmm_softmax_xent_grad_workspace_bytes(d, h, 7)
    assert n > L.gmm_softmax_xent_grad_workspace_bytes(d, h, 1) > 0
    grad = lambda dx, dw, db, lse=E, ws=WS, have=BIG: L.gmm_softmax_xent_grad(d, h, C, lse, None, dx, dw, db, 0, ws, have, None)  # noqa: E731
    assert grad(None, None, None) == INV
    assert grad(F, G_, None, lse=None) == INV
    assert grad(A, None, None) == INV and "overlaps" in last()          # dx on the rows
    assert grad(None, P((2 << 40) + 6), None) == INV                    # dw inside the head
    assert grad(F, F, None) == INV
    assert grad(P((6 << 40) + 1), None, None) == INV                    # misaligned
    for ws, have in ((None, BIG), (P((1 << 50) + 16), BIG), (WS, n - 1)):
        assert grad(F, G_, H, ws=ws, have=have) == WSE


def test_xent_workspaces_are_bounded():
    L = _abi.lib()
    f = lambda N, V: L.gmm_softmax_xent_workspace_bytes(ctypes.byref(rows(N=N)), ctypes.byref(head(V=V)))  # noqa: E731
    assert 0 < f(10 ** 8, 10 ** 5) < 1 << 32
    wide = L.gmm_softmax_xent_workspace_bytes(ctypes.byref(rows(N=10 ** 8, D=256)), ctypes.byref(head(V=10 ** 5, D=256)))
    assert 0 < wide < 1 << 28
    assert f(1, 10 ** 6) < 1 << 20
    # G's pieces: far below N V elements
    g = L.gmm_softmax_xent_grad_workspace_bytes(ctypes.byref(rows(N=10 ** 6)), ctypes.byref(head(V=10 ** 6)), 7)
    assert 0 < g < 4 << 30


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), INV), (dict(N=-1), INV), (dict(N=1 << 31), UNS), (dict(N=1 << 28, m=8), UNS), (dict(idx=None), INV),
    (dict(out=None), INV), (dict(table=dict(N=0)), INV), (dict(table=dict(D=65537)), UNS), (dict(table=dict(x=None)), INV),
    (dict(table=dict(dtype=5)), INV), (dict(table=dict(ld=3)), INV), (dict(out=P((1 << 40) + 64)), INV),
    (dict(out=P((5 << 40) + 1)), INV), (dict(table=dict(Bn=1 << 16, N=1 << 16)), UNS), (dict(out=C), INV),
])
def test_lookup_refusals(kw, status):
    L = _abi.lib()
    a = dict(N=10, m=2, idx=C, w=None, out=F)
    a.update({k: v for k, v in kw.items() if k != "table"})
    t = rows(**{**dict(N=20), **kw.get("table", {})})
    assert L.gmm_codebook_lookup(ctypes.byref(t), a["N"], a["m"], a["idx"], a["w"], 1.0, a["out"], None) == status and last()


def test_lookup_grad_refusals():
    L = _abi.lib()

    def grad(d=None, K=20, m=2, idx=C, w=None, table=None, dt=F, dw=None, ws=WS, have=BIG):
        d = rows(N=10) if d is None else d
        return L.gmm_codebook_lookup_grad(ctypes.byref(d), K, m, idx, w, 1.0, ctypes.byref(table) if table else None, dt, dw,
                                          0, ws, have, None)

    t = rows(N=20, x=B)
    assert grad(K=0) == INV and grad(m=0) == INV and grad(idx=None) == INV and grad(dt=None) == INV
    assert grad(K=1 << 31) == UNS and grad(d=rows(N=1 << 30), m=2) == UNS
    assert grad(dw=G_) == INV and grad(dw=G_, table=rows(N=19, x=B)) == INV
    assert grad(dw=G_, table=rows(N=20, D=32, x=B)) == INV
    assert grad(dw=G_, table=rows(N=20, x=B, dtype=_abi.DT_F32)) == UNS
    assert grad(dt=A) == INV and grad(dt=C) == INV and grad(dt=F, dw=F, table=t) == INV and grad(dw=B, table=t) == INV
    assert grad(dt=P((5 << 40) + 1)) == INV
    n = L.gmm_codebook_lookup_grad_workspace_bytes(ctypes.byref(rows(N=10)), 20, 2)
    assert n > 0
    assert grad(ws=None) == WSE and grad(ws=P((1 << 50) + 8)) == WSE and grad(have=n - 1) == WSE
    assert L.gmm_codebook_lookup_grad_workspace_bytes(ctypes.byref(rows(N=10)), 0, 2) == 0


def test_clip_refusals():
    L = _abi.lib()

    def clip(ts, max_norm=1.0, ws=WS, have=BIG, count=None):
        arr = (_abi.GmmTensor * max(1, len(ts)))(*[_abi.GmmTensor(*t) for t in ts])
        return L.gmm_clip_grad_norm(arr, len(ts) if count is None else count, max_norm, None, ws, have, None)

    a, b, c = 1 << 40, 2 << 40, 3 << 40
    assert clip([]) == INV and L.gmm_clip_grad_norm(None, 1, 1.0, None, WS, BIG, None) == INV
    assert clip([(a, a, 10, 7)]) == INV and clip([(a, a, -1, 0)]) == INV and clip([(None, a, 3, 0)]) == INV
    assert clip([(a, None, 3, 0)]) == INV and clip([(a + 2, a + 2, 3, 0)]) == INV and clip([(a, a, 1 << 40, 0)]) == UNS
    assert clip([(a, a, 10, 0)], max_norm=-1.0) == INV and clip([(a, a, 10, 0)], max_norm=float("nan")) == INV
    # the same tensor twice, an output in another's input, an output shifted over its own input
    assert clip([(a, a, 10, 0), (a, a, 10, 0)]) == INV and "overlaps" in last()
    assert clip([(a, b, 10, 0), (b, c, 10, 0)]) == INV
    assert clip([(a, a + 4, 10, 0)]) == INV
    assert clip([(a, b, 10, 0), (a, b + 36, 10, 0)]) == INV
    assert clip([(a, a, 10, 0)], ws=None) == WSE
    n = L.gmm_clip_grad_norm_workspace_bytes(1)
    assert n > 0 and clip([(a, a, 10, 0)], have=n - 1) == WSE and L.gmm_clip_grad_norm_workspace_bytes(0) == 0


def test_struct_layouts():
    assert ctypes.sizeof(_abi.GmmHead) == 8 + 8 + 2 * 8 + 8
    assert ctypes.sizeof(_abi.GmmTensor) == 8 + 8 + 8 + 8


def test_python_checks_on_the_host():
    """The binding's own checks, with CPU tensors: shapes and types first, then the device."""
    import torch

    import soft_clustering_em_amd as g
    X, W = torch.randn(4, 8), torch.randn(5, 8)
    y = torch.zeros(4, dtype=torch.int32)
    z = torch.zeros(4)
    for bad in (lambda: g.gmm_softmax_xent(X, W, y.long()), lambda: g.gmm_softmax_xent(X, W[:, :7], y),
                lambda: g.gmm_softmax_xent(X.double(), W, y), lambda: g.gmm_softmax_xent(X, W.half(), y),
                lambda: g.gmm_softmax_xent(X, W, y[:3]), lambda: g.gmm_softmax_xent(X.t(), W, y),
                lambda: g.gmm_softmax_xent(X, W, y, bias=torch.zeros(4)), lambda: g.gmm_softmax_xent(X, W, y),
                lambda: g.gmm_softmax_xent_grad(X, W, y, z, accumulate=True),
                lambda: g.gmm_softmax_xent_grad(X, W, y, z[:2]), lambda: g.gmm_softmax_xent_grad(X, W, y, z),
                lambda: g.gmm_codebook_lookup(W, y.long()), lambda: g.gmm_codebook_lookup(W, y, weights=z[:3]),
                lambda: g.gmm_codebook_lookup(W, torch.zeros(1, 2, 3, 4, dtype=torch.int32)), lambda: g.gmm_codebook_lookup(W, y),
                lambda: g.gmm_codebook_lookup_grad(X, y[:3], 5), lambda: g.gmm_codebook_lookup_grad(X, y, 5, table=X),
                lambda: g.gmm_codebook_lookup_grad(X, y, 5, dweights=z), lambda: g.gmm_codebook_lookup_grad(X, y, 5, accumulate=True),
                lambda: g.gmm_codebook_lookup_grad(X, y, 5), lambda: g.gmm_clip_grad_norm([], 1.0),
                lambda: g.gmm_clip_grad_norm([X.t()], 1.0), lambda: g.gmm_clip_grad_norm([X.double()], 1.0),
                lambda: g.gmm_clip_grad_norm([X], 1.0, out=[X, X]), lambda: g.gmm_clip_grad_norm([X], 1.0, out=[W]),
                lambda: g.gmm_clip_grad_norm([X], 1.0)):
        with pytest.raises(ValueError):
            bad()


def test_lookup_refuses_rows_of_more_than_4096_codes():
    L = _abi.lib()
    t = _abi.GmmData(ctypes.c_void_p(256), _abi.DT_F32, 1, 10, 8, 8, 80)
    p = ctypes.c_void_p(4096)
    assert L.gmm_codebook_lookup(ctypes.byref(t), 2, 4097, p, None, 1.0, p, None) == UNS
    assert L.gmm_codebook_lookup_grad(ctypes.byref(t), 5, 4097, p, None, 1.0, None, p, None, 0, p, 1 << 20, None) == UNS
    assert L.gmm_codebook_lookup_grad_workspace_bytes(ctypes.byref(t), 5, 4097) == 0


def _grad_bytes(N, D, V, dtype=_abi.DT_BF16, want=7):
    return _abi.lib().gmm_softmax_xent_grad_workspace_bytes(ctypes.byref(rows(N=N, D=D, dtype=dtype)),
                                                            ctypes.byref(head(V=V, D=D, dtype=dtype)), want)


@pytest.mark.parametrize("want", [1, 2, 4, 7])
@pytest.mark.parametrize("N,D,V,dtype", [(10 ** 6, 768, 16384, _abi.DT_BF16), (1 << 20, 256, 32768, _abi.DT_F32),
                                         (1 << 24, 256, 32768, _abi.DT_BF16), (10 ** 6, 256, 50000, _abi.DT_BF16),
                                         (10 ** 6, 1000, 200, _abi.DT_F16)])
def test_gradient_workspaces_do_not_grow_with_the_rows(N, D, V, dtype, want):
    """Rows in chunks: beside the chunks' parts there is a coefficient per row
    (4 bytes), and one float32 slab of the smaller side where the classes are
    in pieces too."""
    a, b = _grad_bytes(N, D, V, dtype, want), _grad_bytes(2 * N, D, V, dtype, want)
    assert 0 < a < 3 << 30 and 0 < b - a <= 4 * N + 256


@pytest.mark.parametrize("want", [1, 2, 4, 7])
def test_gradient_workspaces_do_not_grow_with_the_classes(want):
    N, D = 40000, 256
    a, b = _grad_bytes(N, D, 10 ** 6, want=want), _grad_bytes(N, D, 8 * 10 ** 6, want=want)
    assert 0 < a == b < 3 << 30
    assert 0 <= _grad_bytes(2 * N, D, 10 ** 6, want=want) - a <= (4 * D + 4) * N + 512


def test_a_stream_of_another_device_is_refused():
    """Two devices are stood in for: the check comes before any call to a GPU."""
    import torch

    from soft_clustering_em_amd import _on

    class On:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

        def get_device(self):
            return self.device.index

    with pytest.raises(ValueError, match="stream"):
        _on(On(1), On(0), None, On(0))
    with pytest.raises(ValueError, match="one GPU"):
        _on(On(0), On(0), On(1))


def test_workspaces_that_count_more_than_they_hold_are_refused():
    import torch

    import soft_clustering_em_amd as g
    X, W, z = torch.randn(4, 8), torch.randn(5, 8), torch.zeros(4)
    y = torch.zeros(4, dtype=torch.int32)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 12, dtype=torch.uint8)[::2]):
        for call in (lambda: g.gmm_softmax_xent(X, W, y, ws=ws), lambda: g.gmm_softmax_xent_grad(X, W, y, z, ws=ws),
                     lambda: g.gmm_codebook_lookup_grad(X, y, 5, ws=ws), lambda: g.gmm_clip_grad_norm([X], 1.0, ws=ws)):
            with pytest.raises(ValueError, match="ws must"):
                call()


def test_clip_refuses_a_norm_on_a_gradient():
    """It would be written before the gradients are read for the scaling."""
    L = _abi.lib()
    a, b = 1 << 40, 2 << 40
    arr = (_abi.GmmTensor * 2)(_abi.GmmTensor(a, b, 10, 0), _abi.GmmTensor(a + 64, a + 64, 10, 1))
    # accepted operands stop at the missing workspace: nothing reaches a GPU
    clip = lambda norm: L.gmm_clip_grad_norm(arr, 2, 1.0, P(norm), None, 0, None)  # noqa: E731
    for at in (a, a + 36, b, b + 36, a + 64, a + 80):
        assert clip(at) == INV and "norm overlaps" in last()
    for at in (a + 40, b + 40, a - 4, a + 84, 3 << 40):
        assert clip(at) == WSE


def test_head_refuses_no_iterations():
    from soft_clustering_em_amd.estimator import SoftmaxHead
    for n in (0, -3):
        with pytest.raises(ValueError, match="max_iter"):
            SoftmaxHead(3, max_iter=n)
