"""gmm_clip_grad_norm against the plain 64-bit form, on the GPU.  The norm is a
float64 sum rounded once: u; an element is a float32 product (2 u: the
coefficient and the product) rounded once to its type."""
import math

import pytest
import torch

import head_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import soft_clustering_em_amd as g
    return g


def make(sizes, types, scale=1.0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def check(grads, outs, norm, max_norm):
    n = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    assert abs(float(norm) - n) <= 2 * ref.U * n
    c = min(1.0, max_norm / (n + 1e-6))
    for i, (a, o) in enumerate(zip(grads, outs)):
        want = a.double() * c
        tol = 3 * ref.U * want.abs()
        ref.within(f"gradient {i}", o, want, tol + ref.half(a.dtype) * (want.abs() + tol) + ref.tiny(a.dtype))


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("sizes,types", [([1], [F32]), ([7], [BF16]), ([8192], [F16]), ([8193, 0, 3], [F32]),
                                         ([5, 1000, 33, 20000, 1, 65536, 8191], [F32, BF16, F16]),
                                         (list(range(1, 150)), [BF16, F32]), ([3_000_001, 17], [BF16, F32]),
                                         ([40_000_003], [F32])])
def test_norm_and_scaling(g, sizes, types, max_norm):
    grads = make(sizes, types)
    outs = [torch.full_like(t, 7) for t in grads]
    kept = [t.clone() for t in grads]
    norm = g.gmm_clip_grad_norm(grads, max_norm, out=outs)
    check(grads, outs, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    same = g.gmm_clip_grad_norm(grads, max_norm)  # in place
    assert torch.equal(norm, same) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_unaligned_views(g):
    big = make([100000], [BF16])[0]
    views = [big[1:5000], big[5003:40001], big[40001:40002], big[50001:99999]]
    kept = [v.clone() for v in views]
    rest = big[40002:50001].clone()
    norm = g.gmm_clip_grad_norm(views, 1.0)
    check(kept, views, norm, 1.0)
    assert torch.equal(big[40002:50001], rest)


def test_squares_outside_float32(g):
    grads = make([1000, 2000], [F32], scale=1e25)
    outs = [torch.empty_like(t) for t in grads]
    check(grads, outs, g.gmm_clip_grad_norm(grads, 1.0, out=outs), 1.0)
    small = make([1000], [F32], scale=1e-30)
    assert float(g.gmm_clip_grad_norm(small, 1.0)) > 0


def test_nan_and_infinite_gradients(g):
    grads = make([100, 200], [F32])
    grads[0][3] = float("inf")
    outs = [torch.empty_like(t) for t in grads]
    assert float(g.gmm_clip_grad_norm(grads, 1.0, out=outs)) == float("inf")
    assert torch.isnan(outs[0][3]) and not outs[1].any() and torch.isnan(outs[0]).sum() == 1
    grads[1][0] = float("nan")
    assert math.isnan(float(g.gmm_clip_grad_norm(grads, 1.0, out=outs)))
    assert all(torch.isnan(o).all() for o in outs)
    zero = [torch.zeros(50, device="cuda")]
    assert float(g.gmm_clip_grad_norm(zero, 1.0)) == 0 and not zero[0].any()


def test_captured(g):
    grads = make([5000, 100, 70000], [F32, BF16])
    outs = [torch.empty_like(t) for t in grads]
    eager = [torch.empty_like(t) for t in grads]
    g.gmm_clip_grad_norm(grads, 1.0, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = g.gmm_clip_grad_norm(grads, 1.0, out=outs)
    for k in range(4):
        for t in grads:
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, g.gmm_clip_grad_norm(grads, 1.0, out=eager)), k
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), k


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 1.0])
def test_no_limit_copies_whatever_the_norm(g, bad):
    grads = make([100, 70000, 7], [F32, BF16, F16])
    grads[0][3] = bad
    kept = [t.clone() for t in grads]
    outs = [torch.empty_like(t) for t in grads]
    for norm in (g.gmm_clip_grad_norm(grads, float("inf"), out=outs), g.gmm_clip_grad_norm(grads, float("inf"))):
        assert math.isfinite(float(norm)) == math.isfinite(bad)
    for k, o, t in zip(kept, outs, grads):
        assert torch.equal(k.view(torch.uint8), o.view(torch.uint8)) and torch.equal(k.view(torch.uint8), t.view(torch.uint8))


@pytest.mark.parametrize("scale,max_norm", [(1e25, 1e-15), (1e25, 1e-30), (1e30, 1e-7), (1.0, 1e-41), (1e-20, 1e-37)])
def test_coefficients_below_float32s_normal_values(g, scale, max_norm):
    grads = make([1000, 20001, 7], [F32, BF16], scale=scale)
    outs = [torch.empty_like(t) for t in grads]
    norm = g.gmm_clip_grad_norm(grads, max_norm, out=outs)
    check(grads, outs, norm, max_norm)
    same = g.gmm_clip_grad_norm(grads, max_norm)  # in place
    assert torch.equal(norm, same) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_thousands_of_tensors(g):
    grads = make([1 + 7 * i % 900 for i in range(3000)], [F32, BF16, F16])
    outs = [torch.empty_like(t) for t in grads]
    check(grads, outs, g.gmm_clip_grad_norm(grads, 1.0, out=outs), 1.0)
