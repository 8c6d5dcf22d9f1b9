"""gmm_route_topm and its gradient against the plain 64-bit form, on the GPU.
Codes are equal; a weight is a float64 value rounded once (u, and 4 ulp of
float64 before it)."""
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


def make(shape, dtype=F32, seed=0, spread=1.5, masked=0.0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = spread * torch.randn(*shape[:-1], shape[-1] + pad, generator=gen, device="cuda")  # noqa: E741
    off = torch.rand(l.shape, generator=gen, device="cuda") < masked
    return l.masked_fill(off, -math.inf).to(dtype)[..., :shape[-1]]


def check(g, logits, m, bias=None, score="softmax", groups=1, keep=None, top=1, renorm=True, scale=1.0, seed=1):
    idx, w = g.gmm_route_topm(logits, m, bias=bias, score=score, groups=groups, keep_groups=keep, group_top=top,
                              renormalize=renorm, scale=scale)
    i_want, w_want = ref.route(logits, m, bias, score, groups, keep, top, renorm, scale)
    assert torch.equal(idx.cpu(), i_want), (idx.cpu() != i_want).nonzero()[:5]
    head_ref.within("weights", w.cpu(), w_want, 1.01 * ref.U * w_want.abs() + 2.0 ** -149)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dw = torch.randn(w.shape, generator=gen, device="cuda")
    ds = torch.randn(logits.shape[-1], generator=gen, device="cuda")
    for a, b in ((dw, None), (None, ds), (dw, ds)):
        dl = g.gmm_route_topm_grad(a, logits, idx, score=score, renormalize=renorm, scale=scale, dscores=b)
        head_ref.within("dlogits", dl.cpu(), *ref.route_grad(a, logits, idx, score, renorm, scale, b))
    return idx, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,E,m", [(1, 1, 1), (5, 2, 2), (3, 8, 3), (100, 16, 4), (67, 60, 6), (64, 64, 8), (33, 65, 16),
                                   (50, 128, 1), (41, 200, 8), (30, 256, 8), (9, 257, 2), (20, 512, 16), (7, 1000, 10),
                                   (5, 1024, 16)])
def test_sizes(g, N, E, m, score, renorm):
    gen = torch.Generator(device="cuda").manual_seed(E)
    check(g, make((N, E), seed=N), m, score=score, renorm=renorm, scale=2.5)
    check(g, make((N, E), seed=N), m, bias=0.1 * torch.randn(E, generator=gen, device="cuda"), score=score, renorm=renorm)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,groups,keep,m", [(256, 8, 4, 8), (64, 64, 20, 16), (60, 4, 1, 5), (36, 6, 6, 3), (1024, 32, 3, 8),
                                             (96, 3, 2, 16), (8, 4, 1, 2), (512, 2, 1, 16)])
def test_groups(g, E, groups, keep, m, top, dtype):
    gen = torch.Generator(device="cuda").manual_seed(E)
    bias = 0.1 * torch.randn(E, generator=gen, device="cuda")
    for b in (None, bias, torch.zeros_like(bias)):  # a zero bias: many equal scores of 16-bit logits
        for score in ("softmax", "sigmoid"):
            check(g, make((40, E), dtype, masked=0.1), m, bias=b, score=score, groups=groups, keep=keep, top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(g, score):
    l = torch.zeros(3, 70, device="cuda")  # noqa: E741
    l[1, 40:50] = 1.0
    l[2, ::7] = -0.0
    for b in (None, torch.zeros(70, device="cuda")):
        idx, w = check(g, l, 8, bias=b, score=score)
        assert idx[0].tolist() == list(range(8)) and idx[1].tolist() == list(range(40, 48))
        check(g, l, 4, bias=b, score=score, groups=7, keep=2, top=2)
        check(g, l, 4, bias=b, score=score, groups=70 // 2, keep=3, top=1)
    # near ties: neighbours in float32, and sums that are equal in float32 and not in float64
    gen = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randint(0, 4, (64, 256), generator=gen, device="cuda").float() * 2.0 ** -22 + 1.0  # noqa: E741
    check(g, l, 8, score=score)
    check(g, l, 8, bias=torch.randint(0, 4, (256,), generator=gen, device="cuda").float() * 2.0 ** -26, score=score, groups=8,
          keep=3, top=2)


def test_switched_off_experts_and_rows(g):
    l = make((6, 40))  # noqa: E741
    l[0] = -math.inf
    l[1, 1:] = float("nan")
    l[2, :37] = -math.inf
    l[3, 5] = math.inf
    l[4] = -3.4e38
    l[4, 7] = float("nan")
    l[5] = torch.finfo(F32).min
    for score in ("softmax", "sigmoid"):
        for b in (None, torch.randn(40, device="cuda") * 0.1):
            for kw in (dict(), dict(groups=8, keep=2, top=2), dict(groups=8, keep=2), dict(renorm=False)):
                idx, w = check(g, l, 5, bias=b, score=score, **kw)
                assert (idx[0] == -1).all() and not w[0].any() and idx[1].tolist() == [0, -1, -1, -1, -1]
                assert torch.isfinite(w).all() and (idx[2] >= 0).sum() <= 3


def test_wide_spreads(g):
    l = make((50, 100), spread=300.0)  # noqa: E741
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check(g, l, 8, score=score, renorm=renorm)
    check(g, l, 8, bias=-l.mean(0) / 100)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strides_and_batches(g, dtype):
    check(g, make((50, 33), dtype, pad=5), 4)
    check(g, make((3, 20, 48), dtype, pad=3), 4, groups=4, keep=2)
    l = make((3, 20, 48), dtype)[:, :11]  # noqa: E741
    check(g, l, 2, score="sigmoid")
    assert g.gmm_route_topm(make((0, 8)), 2)[0].shape == (0, 2)
    assert g.gmm_route_topm_grad(torch.empty(0, 2, device="cuda"), make((0, 8)),
                                 torch.empty(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 8)


def test_gradient_of_foreign_codes(g):
    """Codes as a caller may hold them: the first value outside ends the row, one expert twice."""
    l = make((5, 20))  # noqa: E741
    idx = torch.tensor([[3, 4, -1], [-1, 4, 5], [20, 1, 2], [7, 7, 1], [0, 1 << 30, 2]], dtype=torch.int32, device="cuda")
    dw = torch.randn(5, 3, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dl = g.gmm_route_topm_grad(dw, l, idx, score=score, renormalize=renorm)
            head_ref.within("dlogits", dl.cpu(), *ref.route_grad(dw, l, idx, score, renorm))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(g, score, renorm):
    l = make((6, 30))  # noqa: E741
    idx, w = g.gmm_route_topm(l, 4, score=score, renormalize=renorm)
    dw, ds = torch.randn_like(w), torch.randn(30, device="cuda")
    dl = g.gmm_route_topm_grad(dw, l, idx, score=score, renormalize=renorm, dscores=ds).cpu().double()
    v = torch.randn(6, 30, dtype=torch.float64)

    def loss(x):
        s = torch.from_numpy(ref.scores(x, score)[1])
        sel = s.gather(1, idx.cpu().long())
        if renorm:
            sel = sel / sel.sum(1, keepdim=True)
        return float((sel * dw.cpu().double()).sum() + (s * ds.cpu().double()).sum())

    h = 1e-5
    slope = (loss(l.cpu().double() + h * v) - loss(l.cpu().double() - h * v)) / (2 * h)
    _, tol = ref.route_grad(dw, l, idx, score, renorm, 1.0, ds)
    # differences: h^2 times a third derivative under 1e3, and 1e-13 / h
    assert abs(float((dl * v).sum()) - slope) <= float((tol * v.abs()).sum()) + 1e-6


def test_codes_feed_lists_and_lookup(g):
    l = make((500, 64), BF16)  # noqa: E741
    idx, w = g.gmm_route_topm(l, 4)
    table = torch.randn(64, 32, device="cuda")
    head_ref.within("rows", g.gmm_codebook_lookup(table, idx, weights=w), *head_ref.lookup(table, idx, w))
    offsets, rows, resp = g.gmm_ivf_lists(idx, 64, resp=w)
    counts = torch.bincount(idx.flatten().long(), minlength=64)
    assert torch.equal(offsets.flatten()[1:65] - offsets.flatten()[:64], counts)


def test_captured(g):
    l = make((300, 96))  # noqa: E741
    bias, dw = 0.1 * torch.randn(96, device="cuda"), torch.randn(300, 6, device="cuda")

    def step():
        idx, w = g.gmm_route_topm(l, 6, bias=bias, score="sigmoid", groups=8, keep_groups=3, group_top=2)
        return idx, w, g.gmm_route_topm_grad(dw, l, idx, score="sigmoid")

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        l.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k


def test_more_experts_asked_for_than_there_are(g):
    for E, m in ((1, 4), (3, 16), (20, 16)):
        for b in (None, torch.randn(E, device="cuda")):
            idx, w = check(g, make((9, E)), m, bias=b)
            assert (idx[:, min(E, m):] == -1).all()


def test_more_rows_than_a_launch_takes(g):
    """2^31 threads of a launch are 2^27 rows of 16 lanes: the rows behind them come in a second one."""
    n = (1 << 27) + 37
    l = torch.zeros(n, 2, dtype=BF16, device="cuda")  # noqa: E741
    l[::2, 1] = 1.0
    idx, w = g.gmm_route_topm(l, 1, renormalize=False)
    at = torch.tensor([0, 1, (1 << 27) - 1, 1 << 27, (1 << 27) + 1, n - 2, n - 1], device="cuda")
    i_want, w_want = ref.route(l[at], 1, renorm=False)
    assert torch.equal(idx[at].cpu(), i_want)
    head_ref.within("weights", w[at].cpu(), w_want, 1.01 * ref.U * w_want)
    assert int(idx.sum(dtype=torch.int64)) == (n + 1) // 2
    dl = g.gmm_route_topm_grad(w, l, idx, renormalize=False)
    head_ref.within("dlogits", dl[at].cpu(), *ref.route_grad(w[at], l[at], idx[at], renorm=False))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep,top", [(12, 1, 1, 1), (64, 8, 3, 2), (256, 8, 4, 2), (256, 1, 1, 1), (600, 4, 2, 1)])
def test_a_bias_that_switches_experts_off(g, score, E, groups, keep, top):
    """-inf and NaN biases choose as a bias far below every score does, and +inf as one far above."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn(500, E, generator=gen, device="cuda")  # noqa: E741
    finite = 0.1 * torch.randn(E, generator=gen, device="cuda")
    odd = finite.clone()
    finite[1::4], odd[1::4] = -1e30, -float("inf")
    finite[2::8], odd[2::8] = -1e30, float("nan")
    how = dict(score=score, groups=groups, keep_groups=keep, group_top=top)
    want, got = g.gmm_route_topm(l, 3, bias=finite, **how), g.gmm_route_topm(l, 3, bias=odd, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool(torch.isfinite(got[1]).all())
    finite[7], odd[7] = 1e30, float("inf")
    want, got = g.gmm_route_topm(l, 3, bias=finite, **how), g.gmm_route_topm(l, 3, bias=odd, **how)
    assert bool((got[0][:, 0] == 7).all()) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep,m", [(4, 2, 1, 2), (64, 16, 5, 8), (320, 64, 20, 8)])
def test_biases_that_cancel_within_a_group(g, score, E, groups, keep, m):
    """A group's two best are forced apart by a bias of either sign, so that its
    score is small and each of its terms is not; groups lie 1e-5 apart.  Rows whose
    float64 scores of the last group kept and the first one dropped differ by less
    than 1e-11 (64 units of float64 at the largest bias) may go either way."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    n, gs = 20000, E // groups
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    s = 0.05 * rand(n, groups, gs)
    s[:, :, 0] = 0.35 + 0.2 * rand(n, groups)
    s[:, :, 1] = 0.9 + 1e-5 * (2 * rand(n, groups) - 1) - s[:, :, 0]
    l = (torch.log(s) if score == "softmax" else torch.logit(s)).view(n, E).float()  # noqa: E741
    for by in (1.0, 30.0, 100.0, 1000.0):
        bias = torch.full((groups, gs), -4.0 * by, device="cuda")
        bias[:, 0], bias[:, 1] = by, -by
        bias = bias.view(E)
        idx, _ = g.gmm_route_topm(l, m, bias=bias, score=score, groups=groups, keep_groups=keep, group_top=2)
        t = (torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())) + bias.double()
        value, order = (t.view(n, groups, gs).topk(2, dim=2).values.sum(2)).sort(dim=1, descending=True, stable=True)
        clear = (value[:, keep - 1] - value[:, keep] > 1e-11) & (value[:, :keep].diff(dim=1).abs() > 0).all(1)
        kept = torch.zeros(n, groups, dtype=torch.bool, device="cuda").scatter_(1, order[:, :keep], True)
        t = t.masked_fill(~kept.repeat_interleave(gs, 1), -math.inf)
        best, at = t.sort(dim=1, descending=True, stable=True)
        clear &= (best[:, :m].diff(dim=1).abs() > 1e-11).all(1)
        assert float(clear.double().mean()) > 0.99
        assert torch.equal(idx[clear].long(), at[clear, :m]), (by, int((idx[clear].long() != at[clear, :m]).any(1).sum()))


@pytest.mark.parametrize("E", [20, 300])
def test_gradient_of_codes_that_are_switched_off(g, E):
    """Codes of experts whose logit is NaN or -inf have no weight and no gradient, and the others' is theirs alone."""
    l = make((4, E))  # noqa: E741
    l[0, 3], l[1, 3], l[2, :] = float("nan"), -math.inf, float("nan")
    idx = torch.tensor([[3, 4], [4, 3], [1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    dw = torch.randn(4, 2, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dl = g.gmm_route_topm_grad(dw, l, idx, score=score, renormalize=renorm)
            head_ref.within("dlogits", dl.cpu(), *ref.route_grad(dw, l, idx, score, renorm))
