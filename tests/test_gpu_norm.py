"""gmm_layer_norm and its gradients against the plain 64-bit form, on the GPU."""
import math

import pytest
import torch

import head_ref
import step_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import soft_clustering_em_amd as g
    return g


def make(shape, dtype, affine=None, seed=0, offset=0.0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    D = shape[-1]
    X = (rand(*shape[:-1], D + pad) + offset).to(dtype)[..., :D]
    dout = rand(*shape).to(dtype)
    gamma, beta = (None, None) if affine is None else ((1 + 0.5 * rand(D)).to(affine), rand(D).to(affine))
    return X, dout, gamma, beta


def check(g, X, dout, gamma, beta, eps=1e-5):
    out, mean, rstd = g.gmm_layer_norm(X, gamma, beta, eps=eps)
    want = ref.norm(X, gamma, beta, eps)
    for name, got, (w, tol) in zip(("out", "mean", "rstd"), (out, mean, rstd), want):
        head_ref.within(name, got, w, tol)
    ones = torch.ones(X.shape[-1], device="cuda") if gamma is None else gamma
    grads = g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma=ones)
    for name, got, (w, tol) in zip(("dX", "dgamma", "dbeta"), grads, ref.norm_grad(dout, X, mean, rstd, ones)):
        head_ref.within(name, got, w, tol)
    return out, mean, rstd, grads


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 64), (17, 63), (1, 4096), (300, 128), (130, 129), (33, 512), (77, 1000), (1000, 100),
          (9, 1025), (40, 2048), (6, 2049), (5, 4097), (3, 8192), (4, 8193), (3, 16384), (2, 16385), (2, 32768), (5000, 24)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_of_every_width(g, shape, dtype):
    check(g, *make(shape, dtype, dtype))


@pytest.mark.parametrize("affine", [None, F32, BF16])
@pytest.mark.parametrize("shape", [(2, 50, 96), (3, 1, 777), (1, 1, 16), (4, 7, 2048)])
def test_batches_and_float32_affine(g, shape, affine):
    check(g, *make(shape, BF16, affine, pad=13))


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("D", [64, 515, 3001])
def test_strided_and_unaligned_rows(g, D, pad):
    X, dout, gamma, beta = make((50, D), F16, F16, pad=pad)
    big = torch.randn(2 * 50 * (D + 5) + 1, device="cuda").half()
    dview = big[1:1 + 50 * (D + 5)].view(50, D + 5)[:, :D]  # every row at another offset from 16 bytes
    dview.copy_(dout)
    check(g, X, dview, gamma, beta)
    batch = big[1:1 + 50 * (D + 5)].view(2, 25, D + 5)[:, :20, :D]  # problems further apart than their rows
    check(g, batch, dout.view(2, 25, D)[:, :20].contiguous(), gamma, beta)


@pytest.mark.parametrize("offset", [100.0, -3e4])
def test_rows_far_from_zero(g, offset):
    check(g, *make((60, 300), F32, F32, offset=offset))


def test_constant_rows_and_eps(g):
    X = torch.full((5, 100), 3.7, device="cuda")
    X[1] = 0.0
    out, mean, rstd, _ = check(g, X, torch.randn_like(X), None, None)
    assert torch.isfinite(out).all() and float(out.abs().max()) < 1e-3
    check(g, *make((5, 100), F32, F32), eps=0.0)
    one = torch.randn(4, 1, device="cuda")
    assert torch.equal(g.gmm_layer_norm(one)[0], torch.zeros_like(one))


def test_nan_and_infinite_rows_stay_in_their_row(g):
    X, dout, gamma, beta = make((6, 200), F32, F32)
    X[1, 3], X[4, 199] = float("nan"), float("inf")
    out, mean, rstd = g.gmm_layer_norm(X, gamma, beta)
    bad = torch.isnan(out).any(1)
    assert bad.tolist() == [False, True, False, False, True, False] and torch.isnan(out[1]).all()
    assert math.isnan(float(mean[1])) and math.isnan(float(rstd[1]))
    rows = torch.tensor([0, 2, 3, 5], device="cuda")
    assert torch.equal(out[rows], g.gmm_layer_norm(X[rows].contiguous(), gamma, beta)[0])


def test_long_sums_over_rows(g):
    X, dout, gamma, beta = make((200000, 40), BF16, BF16)
    check(g, X, dout, gamma, beta)


def test_no_rows(g):
    X = torch.empty(0, 16, device="cuda")
    out, mean, rstd = g.gmm_layer_norm(X)
    assert out.shape == (0, 16) and mean.shape == (0,)
    gamma = torch.ones(16, device="cuda")
    dX, dg, db = g.gmm_layer_norm_grad(X, X, mean, rstd, gamma=gamma)
    assert dX.shape == (0, 16) and not dg.any() and not db.any()
    g.gmm_layer_norm_grad(X, X, mean, rstd, gamma=gamma, dX=dX, dgamma=gamma.clone().fill_(2), dbeta=db, accumulate=True)


@pytest.mark.parametrize("shape,dtype", [((70, 200), F32), ((70, 200), BF16), ((3, 20000), F16)])
def test_accumulate_and_left_out(g, shape, dtype):
    X, dout, gamma, beta = make(shape, dtype, dtype)
    _, mean, rstd = g.gmm_layer_norm(X, gamma, beta)
    full = g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma=gamma)
    for i in range(3):
        only = [False] * 3
        only[i] = None
        got = g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma, *only)
        assert [t is not None for t in got] == [k == i for k in range(3)] and torch.equal(got[i], full[i])
    old = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in full]
    bufs = [t.clone() for t in old]
    g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma, *bufs, accumulate=True)
    for name, b, (w, tol) in zip(("dX", "dgamma", "dbeta"), bufs, ref.norm_grad(dout, X, mean, rstd, gamma, old)):
        head_ref.within(name, b, w, tol)


def test_gradient_against_differences(g):
    """Central differences of the 64-bit forward pass along random directions."""
    X, dout, gamma, beta = make((7, 90), F32, F32)
    _, mean, rstd = g.gmm_layer_norm(X, gamma, beta)
    grads = g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma=gamma)
    at = [t.double() for t in (X, gamma, beta)]
    loss = lambda t: float((ref.norm(*t)[0][0] * dout.double()).sum())  # noqa: E731
    for i, got in enumerate(grads):
        for seed in range(3):
            gen = torch.Generator(device="cuda").manual_seed(seed)
            v = torch.randn(at[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            h = 1e-5
            up, down = ([a + s * h * v if k == i else a for k, a in enumerate(at)] for s in (1, -1))
            slope = (loss(up) - loss(down)) / (2 * h)
            # differences: h^2 of the third derivative (under 1e3 here) and 1e-12 / h; the gradient: its own bound
            _, tol = ref.norm_grad(dout, X, mean, rstd, gamma)[i]
            # mean and rstd themselves are rounded: u of the terms
            near = float((tol * v.abs()).sum()) + 100 * ref.U * float((got.double() * v).abs().sum()) + 1e-6 * abs(slope) + 1e-6
            assert abs(float((got.double() * v).sum()) - slope) <= near


def test_captured_and_on_a_stream(g):
    X, dout, gamma, beta = make((500, 384), BF16, BF16)
    s = torch.cuda.Stream()

    def step(**kw):
        out, mean, rstd = g.gmm_layer_norm(X, gamma, beta, **kw)
        return (out, mean, rstd) + g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma=gamma, **kw)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        X.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), k
    want = step()
    torch.cuda.synchronize()
    other = step(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))


def test_more_rows_than_a_launch_takes(g):
    """2^31 threads of a launch are 2^27 rows of 16 threads: the rows behind them come in a second one."""
    n = (1 << 27) + 37
    X = torch.arange(8, device="cuda").to(BF16).expand(n, 8).contiguous()
    X[1 << 27:, 0] = 5.0
    out, _, _ = g.gmm_layer_norm(X, mean=False, rstd=False)
    at = torch.tensor([0, 1, (1 << 27) - 1, 1 << 27, n - 2, n - 1], device="cuda")
    head_ref.within("out", out[at], *ref.norm(X[at])[0])
    assert torch.equal(out[:1000], out[0].expand(1000, 8)) and torch.equal(out[1 << 27:], out[n - 1].expand(37, 8))


def test_rows_behind_those_of_a_launch(g):
    """2^31 threads of a launch are 2^29 rows of 4 lanes (two bf16 values are one piece): the last 37 come in a second one."""
    n = (1 << 29) + 37
    X = torch.zeros(n, 2, dtype=BF16, device="cuda")
    X[:, 1] = 1.0
    X[1 << 29:, 0] = 5.0
    X[n - 1, 0] = -3.0
    mean = torch.zeros(n, device="cuda")
    out, _, _ = g.gmm_layer_norm(X, mean=mean, rstd=False)
    at = torch.tensor([0, 1, (1 << 29) - 1, 1 << 29, (1 << 29) + 1, n - 2, n - 1], device="cuda")
    head_ref.within("out", out[at], *ref.norm(X[at])[0])
    head_ref.within("mean", mean[at], *ref.norm(X[at])[1])
    assert torch.equal(out[:1000], out[0].expand(1000, 2)) and torch.equal(out[(1 << 29) - 1000:1 << 29], out[0].expand(1000, 2))
    assert torch.equal(out[1 << 29:n - 1], out[n - 2].expand(36, 2))


@pytest.mark.parametrize("shape,dtype,offset", [((60, 300), F32, 0.0), ((60, 300), F32, 100.0), ((60, 300), F32, -3e4),
                                                ((4, 9000), F32, 100.0), ((4, 9000), F32, -3e4), ((50, 64), BF16, 3.0)])
def test_gradients_of_rows_far_from_zero(g, shape, dtype, offset):
    """Against 64-bit gradients with their own mean and rstd: beside norm_grad's
    bound, xh is off by what the float32 mean is (half a unit in its last place, and
    the sum's own share) times rstd, and by rstd's own relative error."""
    X, dout, gamma, beta = make(shape, dtype, dtype, offset=offset)
    _, mean, rstd = g.gmm_layer_norm(X, gamma, beta)
    grads = g.gmm_layer_norm_grad(dout, X, mean, rstd, gamma=gamma)
    _, (m, m_tol), (r, r_tol) = ref.norm(X, gamma, beta)
    x, y, q = X.double(), dout.double(), dout.double() * gamma.double()
    m, r = m[:, None], r[:, None]
    xh = (x - m) * r
    off = ((m_tol[:, None] + ref.U * m.abs()) * r + r_tol[:, None] / r * xh.abs()) * 1.01
    a, b = q.mean(1, keepdim=True), (q * xh).mean(1, keepdim=True)
    dX = r * (q - a - xh * b)
    more = r * (off * b.abs() + (xh.abs() + off) * (q.abs() * off).mean(1, keepdim=True)) + r_tol[:, None] * (dX / r).abs() * 1.01
    for name, got, want, extra, (_, tol) in zip(("dX", "dgamma", "dbeta"), grads, (dX, (y * xh).sum(0), y.sum(0)),
                                                (more, (y.abs() * off).sum(0), 0.0), ref.norm_grad(dout, X, mean, rstd, gamma)):
        head_ref.within(name, got, want, tol + 1.01 * extra)
