"""Routing, lookup, layer norm, head, clipping, AdamW and sampling together, as
they are used: a training step of a mixture of codes (expert logits -> weighted
codes -> rows -> normalised rows -> logits over classes), and SoftmaxHead over
them."""
import math

import pytest
import torch

import head_ref
import step_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import soft_clustering_em_amd as g
    return g


def model(N=300, E=24, D=64, V=50, dtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    params = [rand(N, E), rand(E, D), 1 + 0.1 * rand(D), 0.1 * rand(D), rand(V, D) / 8, 0.1 * rand(V)]
    params = [p.to(dtype) if i in (0, 1, 4) else p for i, p in enumerate(params)]
    labels = torch.randint(-1, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    return params, labels


def gradients(g, params, labels, m=4, score="softmax"):
    """The mean loss's parts and the gradients of the expert logits, the table,
    gamma, beta, the head and its bias; and the codes."""
    logits, table, gamma, beta, W, bias = params
    idx, w = g.gmm_route_topm(logits, m, score=score)
    rows = g.gmm_codebook_lookup(table, idx, weights=w)
    x, mean, rstd = g.gmm_layer_norm(rows, gamma, beta)
    loss, lse = g.gmm_softmax_xent(x, W, labels, bias=bias)
    dx, dW, db = g.gmm_softmax_xent_grad(x, W, labels, lse, bias=bias)
    drows, dgamma, dbeta = g.gmm_layer_norm_grad(dx, rows, mean, rstd, gamma=gamma)
    dtable, dw = g.gmm_codebook_lookup_grad(drows, idx, table.shape[0], table=table, weights=w)
    dlogits = g.gmm_route_topm_grad(dw, logits, idx, score=score)
    return loss, [dlogits, dtable, dgamma, dbeta, dW, db], idx


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_of_the_whole_step(g, score):
    """Against automatic differentiation in 64 bits.  Each of the six stages adds
    relative errors of at most u times its longest chain of additions (100) to
    values whose absolute sums are up to 8 times the sums: 6 * 100 * 8 u = 3e-4 of a
    gradient's norm."""
    params, labels = model()
    loss, grads, idx = gradients(g, params, labels, score=score)
    p = [t.double().requires_grad_() for t in params]
    s = torch.softmax(p[0], 1) if score == "softmax" else torch.sigmoid(p[0])
    sel = s.gather(1, idx.long())
    w = sel / sel.sum(1, keepdim=True)
    rows = (w[..., None] * p[1][idx.long()]).sum(1)
    d = rows - rows.mean(1, keepdim=True)
    x = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * p[2] + p[3]
    z = x @ p[4].t() + p[5]
    live = labels >= 0
    want = (torch.logsumexp(z, 1) - z.gather(1, labels.clamp_min(0).long()[:, None])[:, 0]) * live
    want.sum().backward()
    assert float((loss.double() - want.detach()).abs().max()) <= 4800 * ref.U * float(want.abs().max())
    for name, got, t in zip(("logits", "table", "gamma", "beta", "head", "bias"), grads, p):
        off = float((got.double() - t.grad).norm() / t.grad.norm())
        assert off <= 4800 * ref.U, (name, off)


def train(g, params, grads, state, step, **kw):
    norm = g.gmm_clip_grad_norm(grads, math.inf)
    g.gmm_adamw_step(params, grads, step=step, lr=0.01, norm=norm, max_norm=0.5, seed=1, **state, **kw)
    return norm


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_captured_beside_eager_steps(g, dtype, bits):
    params, labels = model(dtype=dtype)
    start = [t.clone() for t in params]
    loss, grads, _ = gradients(g, params, labels)
    train(g, params, grads, g.new_adamw_state(params, bits), 1)  # buffers and kernels in place before the capture
    for p, s in zip(params, start):
        p.copy_(s)
    state, count = g.new_adamw_state(params, bits), torch.ones(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads, _ = gradients(g, params, labels)
        norm = train(g, params, grads, state, count)
        tokens, _ = g.gmm_sample(params[0], torch.full((300,), 0.3, device="cuda"), top_k=8, top_p=0.9)
        count.add_(1)
    other, other_state = [t.clone() for t in start], g.new_adamw_state(start, bits)
    for step in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        want_loss, want_grads, _ = gradients(g, other, labels)
        want_norm = train(g, other, want_grads, other_state, step)
        want_tokens, _ = g.gmm_sample(other[0], torch.full((300,), 0.3, device="cuda"), top_k=8, top_p=0.9)
        assert torch.equal(loss, want_loss) and torch.equal(norm, want_norm) and torch.equal(tokens, want_tokens), step
        for a, b in zip(params + grads + state["m"] + state["v"], other + want_grads + other_state["m"] + other_state["v"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), step
    assert all(torch.isfinite(t).all() for t in params)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("norm", [None, 0.05])
def test_head_fit_with_adamw(g, bits, norm):
    """fit is the calls that it is documented to make."""
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(1500, 24, generator=gen, device="cuda")
    y = torch.randint(-1, 7, (1500,), generator=gen, device="cuda", dtype=torch.int32)
    kw = dict(learning_rate=0.02, optimizer="adamw", weight_decay=0.1, state_bits=bits, layer_norm=True, max_grad_norm=norm,
              random_state=3)
    head = SoftmaxHead(7, max_iter=4, **kw).fit(X, y)
    assert head.n_iter_ == 4 and len(head.loss_history_) == 4 and (head.grad_norm_ is None) == (norm is None)
    mine = SoftmaxHead(7, **kw)._set(torch.zeros(7, 24, device="cuda"), torch.zeros(7, device="cuda"))
    mine._ready()
    params = mine._parameters()
    state = g.new_adamw_state(params, bits)
    for step in range(1, 5):
        _, *grads = mine.loss_and_gradients(X, y)
        n = None if norm is None else g.gmm_clip_grad_norm([t.clone() for t in grads], math.inf)
        g.gmm_adamw_step(params, grads, step=step, lr=0.02, weight_decay=[0.1, 0.0, 0.0, 0.0], norm=n, max_norm=norm, seed=3, **state)
    for a, b in zip(head._parameters(), params):
        assert torch.equal(a, b)


def test_head_gradients_with_layer_norm(g):
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(4)
    for dtype in (torch.float32, torch.float16):
        X = (3 + torch.randn(700, 32, generator=gen, device="cuda")).to(dtype)
        y = torch.randint(-1, 9, (700,), generator=gen, device="cuda", dtype=torch.int32)
        head = SoftmaxHead(9, layer_norm=True)._set(torch.randn(9, 32, generator=gen, device="cuda"), torch.randn(9, device="cuda"))
        loss, *grads = head.loss_and_gradients(X, y)
        p = [t.double().requires_grad_() for t in head._parameters()]
        x = torch.nn.functional.layer_norm(X.double(), (32,), p[2], p[3], 1e-5)
        z = x @ p[0].t() + p[1]
        live = y >= 0
        want = ((torch.logsumexp(z, 1) - z.gather(1, y.clamp_min(0).long()[:, None])[:, 0]) * live).sum() / live.sum()
        want.backward()
        assert abs(float(loss) - float(want)) <= 3200 * ref.U * float(want)
        for got, t in zip(grads, p):  # four stages, as above
            assert float((got.double() - t.grad).norm() / t.grad.norm()) <= 3200 * ref.U
        assert abs(head.score(X, y) + float(want)) <= 3200 * ref.U * float(want)


def test_head_routes_and_samples(g):
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(400, 16, generator=gen, device="cuda")
    head = SoftmaxHead(30)._set(torch.randn(30, 16, generator=gen, device="cuda"), torch.zeros(30, device="cuda"))
    logits = head.logits(X)
    want = X.double() @ head.coef_.double().t()
    assert float((logits.double() - want).abs().max()) <= 20 * ref.U * float((X.double().abs() @ head.coef_.double().abs().t()).max())
    idx, w = head.route(X, 4, score="sigmoid", scale=2.0)
    i_want, w_want = ref.route(logits, 4, score="sigmoid", scale=2.0)
    assert torch.equal(idx.cpu(), i_want)
    head_ref.within("weights", w.cpu(), w_want, 1.01 * ref.U * w_want)
    u = torch.rand(400, generator=gen, device="cuda")
    classes, logp = head.sample(X, temperature=0.7, top_k=10, u=u)
    same, _ = g.gmm_sample(logits, u, temperature=0.7, top_k=10)
    assert torch.equal(classes, same) and (logp <= 0).all()
    assert torch.equal(head.sample(X)[0], head.sample(X)[0])
    assert torch.equal(head.sample(X, temperature=0.0)[0].long(), logits.argmax(1))


def test_refusals_on_the_gpu(g):
    from soft_clustering_em_amd.estimator import SoftmaxHead
    X, z = torch.randn(4, 8, device="cuda"), torch.zeros(4, device="cuda")
    v, idx = torch.ones(8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    st = g.new_adamw_state([X])
    for bad in (lambda: g.gmm_layer_norm(X, v.cpu()), lambda: g.gmm_layer_norm(X, out=X.cpu()),
                lambda: g.gmm_layer_norm_grad(X.cpu(), X, z, z), lambda: g.gmm_route_topm(X, 2, bias=v.cpu()),
                lambda: g.gmm_route_topm_grad(torch.zeros(4, 2), X, idx), lambda: g.gmm_sample(X, z.cpu()),
                lambda: g.gmm_sample(X, z, top_p=z.cpu()), lambda: g.gmm_adamw_step([X], [X.cpu()], step=1, **st),
                lambda: g.gmm_adamw_step([X], [X.clone()], step=torch.ones(1, dtype=torch.int64), **st),
                lambda: SoftmaxHead(3, optimizer="sgd"), lambda: SoftmaxHead(3, state_bits=16), lambda: SoftmaxHead(3, weight_decay=0.1)):
        with pytest.raises(ValueError):
            bad()
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    for bad in (lambda: g.gmm_layer_norm(X, out=X), lambda: g.gmm_layer_norm_grad(X, X, z, z, gamma=v, ws=small),
                lambda: g.gmm_route_topm(X, 17), lambda: g.gmm_route_topm(X, 2, groups=3), lambda: g.gmm_sample(X, z, temperature=-1.0),
                lambda: g.gmm_sample(X, z, ws=small), lambda: g.gmm_sample(X, z, top_p=math.nan),
                lambda: g.gmm_adamw_step([X], [X], step=1, **st), lambda: g.gmm_adamw_step([X], [X.clone()], step=0, **st),
                lambda: g.gmm_adamw_step([X, X], [X.clone(), X.clone()], st["m"] * 2, st["v"] * 2, 1)):
        with pytest.raises(g.GmmError):
            bad()
    for bad in (lambda: SoftmaxHead(3).sample(X), lambda: SoftmaxHead(3).route(X)):
        with pytest.raises(RuntimeError):
            bad()


@pytest.mark.parametrize("layer_norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_a_draw_has_the_probability_that_log_proba_gives(g, dtype, layer_norm):
    """The head of bfloat16 rows is rounded to their type in both.  A logit is a sum
    of 40 products in float32 in any order, the loss's bound beside it."""
    from soft_clustering_em_amd.estimator import SoftmaxHead
    gen = torch.Generator(device="cuda").manual_seed(6)
    X = torch.randn(500, 40, generator=gen, device="cuda").to(dtype)
    head = SoftmaxHead(30, layer_norm=layer_norm)._set(torch.randn(30, 40, generator=gen, device="cuda"),
                                                       torch.randn(30, generator=gen, device="cuda"))
    u = torch.rand(500, generator=gen, device="cuda")
    classes, logp = head.sample(X, u=u)
    want = head.log_proba(X, classes)
    size = float((head._rows(head._check(X, classes)).double().abs() @ head.coef_.double().abs().t()).max()) + 4.0
    # both sides' logits (44 roundings), and log-sum-exps and differences (300)
    assert float((logp.double() - want.double()).abs().max()) <= 2 * 44 * ref.U * size + 300 * ref.U * (size + 8)
