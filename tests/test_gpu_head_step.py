"""The softmax head, the codebook and the clipping together, as they are used:
a training step of a model that predicts the next code (codes -> rows of a
table -> logits over the same table), and the estimators over them."""
import math

import numpy as np
import pytest
import torch

import head_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import soft_clustering_em_amd as g
    return g


def step(g, table, codes, labels, bias, gloss, max_norm):
    """One step's gradients: the table's (from both of its uses) and the bias's, clipped."""
    rows = g.gmm_codebook_lookup(table, codes, scale=2.0)
    loss, lse = g.gmm_softmax_xent(rows, table, labels, bias=bias)
    dX, dW, db = g.gmm_softmax_xent_grad(rows, table, labels, lse, gloss=gloss, bias=bias)
    g.gmm_codebook_lookup_grad(dX, codes, table.shape[0], scale=2.0, dtable=dW, accumulate=True)
    norm = g.gmm_clip_grad_norm([dW, db], max_norm)
    return loss, dW, db, norm


@pytest.mark.parametrize("N,D,K", [(300, 48, 90), (1000, 200, 333), (40, 64, 1000)])
def test_next_code_step(g, N, D, K):
    """Against autograd in 64 bits.  The bound: the head's (head_ref, with the
    rows' gradient carried through the lookup) -- dX's bound summed over the
    codes' rows, three more float32 operations an entry, and the clipping's."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    table = torch.randn(K, D, generator=gen, device="cuda") / D ** 0.5
    codes = torch.randint(0, K, (N,), generator=gen, device="cuda", dtype=torch.int32)
    labels = torch.randint(-1, K, (N,), generator=gen, device="cuda", dtype=torch.int32)
    bias = torch.randn(K, generator=gen, device="cuda")
    gloss = torch.rand(N, generator=gen, device="cuda")
    loss, dT, db, norm = step(g, table, codes, labels, bias, gloss, 0.5)

    t, b = (x.double().requires_grad_() for x in (table, bias))
    logits = (2.0 * t[codes.long()]) @ t.t() + b
    live = labels >= 0
    want = (torch.logsumexp(logits, 1) - logits.gather(1, labels.clamp_min(0).long()[:, None])[:, 0]) * live
    (want * gloss.double()).sum().backward()
    rows = g.gmm_codebook_lookup(table, codes, scale=2.0)
    exact, tol = ref.xent(rows, table, labels, bias, gloss)  # the rows are exact: a power of two times a row
    ref.within("loss", loss, want.detach(), tol["loss"])
    n = math.sqrt(float((t.grad ** 2).sum() + (b.grad ** 2).sum()))
    # the table's bound before clipping
    carried = torch.zeros(K, D, dtype=torch.float64, device="cuda").index_add_(0, codes.long(), 2.0 * tol["dX"])
    size = torch.zeros_like(carried).index_add_(0, codes.long(), 2.0 * exact["dX"].abs())
    t_tol = tol["dW"] + carried + (N + 8) * ref.U * (size + t.grad.abs())
    slack = math.sqrt(float((t_tol ** 2).sum() + (tol["db"] ** 2).sum()))  # how far the norm may be off
    assert abs(float(norm) - n) <= slack + 4 * ref.U * n
    c = min(1.0, 0.5 / (n + 1e-6))
    rel = slack / n + 8 * ref.U
    ref.within("table", dT, c * t.grad, c * t_tol * 1.01 + rel * (c * t.grad).abs())
    ref.within("bias", db, c * b.grad, c * tol["db"] * 1.01 + rel * (c * b.grad).abs())


def test_step_captured_beside_eager_steps(g):
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(500, 96, generator=gen, device="cuda").bfloat16()
    codes = torch.randint(0, 500, (700,), generator=gen, device="cuda", dtype=torch.int32)
    labels = torch.randint(0, 500, (700,), generator=gen, device="cuda", dtype=torch.int32)
    bias = torch.randn(500, generator=gen, device="cuda")
    args = (table, codes, labels, bias, None, 1.0)
    step(g, *args)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:  # two graphs of the same tensors, each with workspaces of its own
        with torch.cuda.graph(graph):
            outs.append(step(g, *args))
    for k in range(3):
        table.normal_()
        codes.copy_(codes.flip(0))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(outs[0], outs[1], step(g, *args)):
            assert torch.equal(a, c) and torch.equal(b, c), k


def test_calls_on_two_streams(g):
    X = torch.randn(3000, 72, device="cuda")
    W = torch.randn(400, 72, device="cuda") / 8
    y = torch.randint(0, 400, (3000,), device="cuda", dtype=torch.int32)
    want = g.gmm_softmax_xent(X, W, y)
    wg = g.gmm_softmax_xent_grad(X, W, y, want[1])
    wt = g.gmm_codebook_lookup_grad(X, y, 400)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            loss, lse = g.gmm_softmax_xent(X, W, y, stream=s)
            got.append((loss, lse) + g.gmm_softmax_xent_grad(X, W, y, lse, stream=s)[:2]
                       + g.gmm_codebook_lookup_grad(X, y, 400, stream=s)[:1])
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, (want[0], want[1], wg[0], wg[1], wt)):
            assert torch.equal(a, b)


def test_head_is_the_posterior_of_a_shared_variance_mixture(g):
    """log_proba of the converted head against the mixture's log responsibilities
    in 64 bits: the head's parameters are rounded to float32, so its logits are
    off by at most u (|W| |x| + |b|) each, beside the call's own bound."""
    from soft_clustering_em_amd.estimator import GaussianMixture, SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(2000, 16, generator=gen, device="cuda") + 3 * torch.randint(0, 3, (2000, 1), generator=gen, device="cuda")
    gm = GaussianMixture(6, "spherical", max_iter=5).fit(X)
    head = SoftmaxHead.from_mixture(gm, variance=1.7)
    y = torch.randint(0, 6, (2000,), generator=gen, device="cuda", dtype=torch.int32)
    mu, w, x = gm.means_.double(), gm.weights_.double(), X.double()
    L = w.log() - ((x[:, None, :] - mu) ** 2).sum(-1) / (2 * 1.7)
    want = (L - torch.logsumexp(L, 1, keepdim=True)).gather(1, y.long()[:, None])[:, 0]
    _, tol = ref.xent(X, head.coef_, y, head.intercept_)
    wnorm = mu.abs() / 1.7
    off = 4 * ref.U * (x.abs() @ wnorm.t() + (w.log().abs() + (mu * mu).sum(1) * 18 / (2 * 1.7))).max(1).values
    ref.within("log_proba", head.log_proba(X, y), want, tol["loss"] + 2 * off)
    assert abs(head.score(X, y) - float(want.mean())) <= float((tol["loss"] + 2 * off).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_fit_runs_and_its_gradients(g, dtype):
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(1500, 24, generator=gen, device="cuda").to(dtype)
    y = torch.randint(-1, 7, (1500,), generator=gen, device="cuda", dtype=torch.int32)
    head = SoftmaxHead(7, max_iter=4, max_grad_norm=0.01, learning_rate=0.5).fit(X, y)
    assert len(head.loss_history_) == head.n_iter_ == 4 and head.loss_history_[0] == pytest.approx(math.log(7), rel=1e-6)
    assert head.coef_.shape == (7, 24) and head.grad_norm_.shape == (1,)
    loss, dW, db = head.loss_and_gradients(X, y)
    n = int((y >= 0).sum())
    want, tol = ref.xent(X, head.coef_.to(dtype), y, head.intercept_, torch.full((1500,), 1.0 / n, device="cuda"))
    ref.within("dW", dW, want["dW"], tol["dW"] + 4 * ref.U * want["dW"].abs())
    ref.within("db", db, want["db"], tol["db"] + 4 * ref.U * want["db"].abs())
    assert abs(float(loss) - float(want["loss"].sum() / n)) <= float(tol["loss"].sum() / n) + 1500 * ref.U * float(loss)


def test_reconstruct(g):
    from soft_clustering_em_amd.estimator import GaussianMixture, KMeans
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(3000, 20, generator=gen, device="cuda")
    km = KMeans(12, max_iter=4).fit(X)
    assert torch.equal(km.reconstruct(km.labels_), km.cluster_centers_[km.labels_.long()])
    gm = GaussianMixture(8, "diag", max_iter=3).fit(X)
    idx, resp, _ = gm.predict_proba_topm(X, 3, 0.05)
    ref.within("rows", gm.reconstruct(X, 3, 0.05), *ref.lookup(gm.means_, idx, resp))


def test_refusals_on_the_gpu(g):
    from soft_clustering_em_amd.estimator import KMeans, SoftmaxHead
    X = torch.randn(5, 8, device="cuda")
    W = torch.randn(3, 8, device="cuda")
    y = torch.zeros(5, dtype=torch.int32, device="cuda")
    _, lse = g.gmm_softmax_xent(X, W, y)
    for bad in (lambda: g.gmm_softmax_xent(X, W.cpu(), y), lambda: g.gmm_softmax_xent(X, W, y.cpu()),
                lambda: g.gmm_codebook_lookup(W, y.cpu()), lambda: g.gmm_clip_grad_norm([X, W.cpu()], 1.0),
                lambda: g.gmm_codebook_lookup_grad(X, y, 3, table=W.cpu(), weights=torch.ones(5, device="cuda")),
                lambda: SoftmaxHead(3).fit(X, y.long()), lambda: SoftmaxHead(3).fit(X[0], y), lambda: SoftmaxHead(0),
                lambda: SoftmaxHead(3, max_grad_norm=0.0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.gmm_softmax_xent_grad(X, W, y, lse, dX=X), lambda: g.gmm_softmax_xent(X, W, y, loss=lse, lse=lse),
                lambda: g.gmm_softmax_xent(X, W, y, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: g.gmm_codebook_lookup(W, y, out=X) if X.data_ptr() == W.data_ptr() else g.gmm_clip_grad_norm([X, X], 1.0),
                lambda: g.gmm_clip_grad_norm([X], float("nan")), lambda: g.gmm_clip_grad_norm([X], -1.0)):
        with pytest.raises(g.GmmError):
            bad()
    for bad in (lambda: SoftmaxHead(3).score(X, y), lambda: KMeans(2).reconstruct(y)):
        with pytest.raises(RuntimeError):
            bad()


def test_head_of_half_rows_keeps_small_gradients(g):
    """Confident rows: the gradients of the other classes are about exp(-25) of
    a row, far below half's spacing, and come inside float32's bound."""
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(1500, 24, generator=gen, device="cuda").half()
    y = torch.zeros(1500, dtype=torch.int32, device="cuda")
    coef = torch.randn(2000, 24, generator=gen, device="cuda") * 0.1
    b = torch.zeros(2000, device="cuda")
    b[0] = 25.0
    loss, dW, db = SoftmaxHead(2000)._set(coef, b).loss_and_gradients(X, y)
    want, tol = ref.xent(X.float(), coef, y, b, torch.full((1500,), 1.0 / 1500, device="cuda"))
    assert 0 < float(want["dW"][1:].abs().max()) < 6e-8
    ref.within("dW", dW, want["dW"], tol["dW"] + 4 * ref.U * want["dW"].abs())
    ref.within("db", db, want["db"], tol["db"] + 4 * ref.U * want["db"].abs())


def test_head_of_half_rows_with_coefficients_past_half(g):
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(700, 40, generator=gen, device="cuda").half()
    y = torch.randint(-1, 20, (700,), generator=gen, device="cuda", dtype=torch.int32)
    coef, b = torch.randn(20, 40, generator=gen, device="cuda") * 1e6, torch.zeros(20, device="cuda")
    head = SoftmaxHead(20)._set(coef, b)
    want, tol = ref.xent(X.float(), coef, y, b)
    ref.within("log_proba", -head.log_proba(X, y), want["loss"], tol["loss"])
    assert math.isfinite(head.score(X, y)) and all(torch.isfinite(t).all() for t in head.loss_and_gradients(X, y))


def test_head_fit_of_half_rows_is_the_fit_of_the_same_float32_rows(g):
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(6)
    X = torch.randn(900, 24, generator=gen, device="cuda").half()
    y = torch.randint(-1, 300, (900,), generator=gen, device="cuda", dtype=torch.int32)
    a, b = (SoftmaxHead(300, max_iter=3, max_grad_norm=0.01).fit(rows, y) for rows in (X, X.float()))
    assert torch.equal(a.coef_, b.coef_) and torch.equal(a.intercept_, b.intercept_)
    assert torch.equal(a.grad_norm_, b.grad_norm_) and a.loss_history_ == b.loss_history_
