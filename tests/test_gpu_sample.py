"""gmm_sample against the plain form with exact integer sums, on the GPU.  Tokens
are equal wherever no threshold lies nearer to a sum than the exponential's own
error moves it; logp is a float64 value (off by 1e-9 at most: the weights'
rounding) rounded once."""
import math

import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import soft_clustering_em_amd as g
    return g


def make(shape, dtype=F32, seed=0, spread=2.5, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = (spread * torch.randn(*shape[:-1], shape[-1] + pad, generator=gen, device="cuda")).to(dtype)[..., :shape[-1]]  # noqa: E741
    return l, torch.rand(shape[:-1], generator=gen, device="cuda")


def check(g, logits, u, unsure=0.02, **kw):
    tokens, logp = g.gmm_sample(logits, u, **kw)
    rows, us = logits.double().cpu().numpy().reshape(-1, logits.shape[-1]), u.double().cpu().numpy().reshape(-1)
    tok, lp = tokens.cpu().numpy().reshape(-1), logp.double().cpu().numpy().reshape(-1)
    skipped = 0
    for r, row in enumerate(rows):
        one = {k: v.cpu().numpy().reshape(-1)[r].item() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
        want, want_lp, sure = ref.sample(row, float(us[r]), **one)
        if not sure:
            skipped += 1
            continue
        assert tok[r] == want, (r, one, int(tok[r]), want)
        assert lp[r] == want_lp or abs(lp[r] - want_lp) <= 2 * ref.U * abs(want_lp) + 1e-9, (r, lp[r], want_lp)
    assert skipped <= unsure * len(rows)
    return tokens, logp


FILTERS = [dict(), dict(temperature=0.0), dict(temperature=0.6), dict(top_k=1), dict(top_k=5), dict(top_k=50, top_p=0.9),
           dict(top_p=0.9), dict(top_p=0.1, temperature=2.0), dict(top_p=0.999), dict(min_p=0.1), dict(min_p=1.0), dict(min_p=7.0),
           dict(top_p=0.0), dict(top_p=-1.0), dict(top_k=10 ** 9, top_p=0.5, min_p=0.01, temperature=1.3), dict(top_k=3, min_p=0.5),
           dict(top_k=700, top_p=0.99)]


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("N,V", [(40, 1), (40, 2), (40, 33), (20, 1000), (8, 5003)])
def test_sizes(g, N, V, kw):
    l, u = make((N, V), seed=V)  # noqa: E741
    check(g, l, u, **kw)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kw", FILTERS)
def test_16_bit_logits(g, kw, dtype):
    """Many equal logits: ties at every threshold."""
    l, u = make((12, 3001), dtype, pad=7)  # noqa: E741
    check(g, l, u, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.9, temperature=0.7), dict(top_k=20000), dict(top_p=0.999),
                                dict(min_p=0.02)])
@pytest.mark.parametrize("V,dtype", [(131072, BF16), (50001, F32), (262144, F16)])
def test_vocabularies(g, V, dtype, kw):
    l, u = make((3, V), dtype)  # noqa: E741
    check(g, l, u, unsure=0.34, **kw)


@pytest.mark.parametrize("kw", FILTERS)
def test_equal_and_few_distinct_logits(g, kw):
    l, u = make((6, 10000))  # noqa: E741
    l[0] = 3.0
    l[1] = torch.where(torch.arange(10000, device="cuda") % 2 == 0, 1.0, 2.0)
    l[2] = -1e30
    l[3] = 0.0
    l[3, 9999] = 50.0
    l[4] = l[4].round()
    l[5] = torch.linspace(0, 1e-5, 10000, device="cuda")
    check(g, l, u, unsure=0.17, **kw)


@pytest.mark.parametrize("kw", FILTERS)
def test_masked_infinite_and_nan_logits(g, kw):
    l, u = make((8, 300))  # noqa: E741
    l[0] = -math.inf
    l[1] = float("nan")
    l[2, :299] = -math.inf
    l[3, ::2] = float("nan")
    l[4, 7] = math.inf
    l[5, 3:5] = math.inf
    l[6] = torch.finfo(F32).min
    l[6, 1::3] = -math.inf
    l[7] = torch.randn(300, device="cuda") * 1e38
    tokens, logp = check(g, l, u, **kw)
    assert tokens[:2].tolist() == [-1, -1] and logp[:2].tolist() == [-math.inf] * 2 and int(tokens[2]) == 299


def test_numbers_at_and_outside_the_ends(g):
    l, _ = make((1, 500))  # noqa: E741
    u = torch.tensor([0.0, -1.0, 1.0, 2.0, float("nan"), 1 - 2.0 ** -24, math.inf, 0.5], device="cuda")
    l = l.expand(8, 500).contiguous()  # noqa: E741
    tokens, _ = check(g, l, u, top_p=0.8)
    assert len(set(tokens[[0, 1, 4]].tolist())) == 1 and len(set(tokens[[2, 3, 5, 6]].tolist())) == 1


def test_settings_of_every_row(g):
    l, u = make((60, 2000))  # noqa: E741
    i = torch.arange(60, device="cuda")
    kw = dict(temperature=torch.tensor([0.0, 0.5, 1.0, -1.0, float("nan")], device="cuda")[i % 5],
              top_k=torch.tensor([0, 1, 7, 5000, -3], dtype=torch.int32, device="cuda")[i % 4],
              top_p=torch.tensor([1.0, 0.5, 0.95], device="cuda")[i % 3],
              min_p=torch.tensor([0.0, 0.2], device="cuda")[i % 2])
    check(g, l, u, **{k: v.contiguous() for k, v in kw.items()})
    check(g, l.view(3, 20, 2000), u.view(3, 20), top_k=kw["top_k"].view(3, 20).contiguous(), top_p=0.9)


def test_frequencies_are_the_probabilities(g):
    """A stratified u = (i + 0.5) / n gives every token its share to within 1 / n."""
    l = torch.tensor([0.0, 1.0, -0.5, 2.0, 0.3], device="cuda")  # noqa: E741
    n = 10000
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens, _ = g.gmm_sample(l.expand(n, 5).contiguous(), u, temperature=0.8)
    p = torch.softmax(l.double() / 0.8, 0)
    share = torch.bincount(tokens.long(), minlength=5).double() / n
    assert float((share - p).abs().max()) <= 1.5 / n


def test_strides_no_rows_and_outputs(g):
    l, u = make((5, 7, 99), BF16, pad=3)  # noqa: E741
    tokens, logp = check(g, l, u, top_p=0.9)
    t2 = torch.empty(5, 7, dtype=torch.int32, device="cuda")
    assert g.gmm_sample(l, u, top_p=0.9, tokens=t2, logp=False)[1] is None and torch.equal(t2, tokens)
    big = torch.randn(20 * 1001 + 3, device="cuda").half()
    for off in (1, 2, 3):
        check(g, big[off:off + 20 * 1001].view(20, 1001)[:, :1000], torch.rand(20, device="cuda"), top_k=30)
    assert g.gmm_sample(torch.empty(0, 9, device="cuda"), torch.empty(0, device="cuda"))[0].shape == (0,)


def test_captured_and_on_two_streams(g):
    l, u = make((30, 20000), BF16)  # noqa: E741
    step = lambda **kw: g.gmm_sample(l, u, temperature=0.8, top_k=40, top_p=0.9, **kw)  # noqa: E731
    step()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    for k in range(4):
        l.normal_()
        u.uniform_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want)), k
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))


def test_one_row_does_not_depend_on_its_batch(g):
    l, u = make((300, 7001), F16)  # noqa: E741
    for kw in (dict(top_p=0.95), dict(top_k=100, min_p=0.01), dict()):
        tokens, logp = g.gmm_sample(l, u, **kw)
        for r in (0, 137, 299):
            t, p = g.gmm_sample(l[r:r + 1], u[r:r + 1], **kw)
            assert t.item() == tokens[r].item() and p.item() == logp[r].item()


def test_reference_on_the_host():
    """The oracle's own tokens against plain float64 probabilities."""
    rng = np.random.default_rng(0)
    for _ in range(50):
        row = rng.normal(size=40) * 2
        t, lp, _ = ref.sample(row, 0.37, top_p=0.8)
        p = np.exp(row - row.max())
        p /= p.sum()
        order = np.argsort(-p, kind="stable")
        keep = order[:1 + int((np.cumsum(p[order]) < 0.8).sum())]
        q = np.zeros(40)
        q[keep] = p[keep] / p[keep].sum()
        assert t == int(np.searchsorted(np.cumsum(q), 0.37, side="right")) and abs(lp - math.log(q[t])) < 1e-9


@pytest.mark.parametrize("kw", FILTERS)
def test_long_rows_of_equal_few_and_masked_logits(g, kw):
    """Rows in parts: equal logits, two values, one live element, dead parts, infinities."""
    V = 40003
    l, u = make((7, V))  # noqa: E741
    l[0] = 3.0
    l[1] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 1.0, 2.0)
    l[2] = -math.inf
    l[2, V - 1] = -7.0
    l[3, :20000] = -math.inf
    l[4] = l[4].round()
    l[5, 35001] = math.inf
    l[5, ::3] = float("nan")
    l[6] = -math.inf
    tokens, logp = check(g, l, u, unsure=0.15, **kw)
    assert int(tokens[2]) == V - 1 and int(tokens[6]) == -1 and float(logp[6]) == -math.inf


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("V,dtype", [(5, F32), (2049, BF16), (20001, F16), (32768, F32)])
def test_many_rows_and_few(g, V, dtype, kw):
    """300 rows in one call and by 100: the same tokens and logarithms."""
    l, u = make((300, V), dtype, seed=V)  # noqa: E741
    l[7] = 1.0
    l[8, ::2] = -math.inf
    tokens, logp = g.gmm_sample(l, u, **kw)
    for i in range(0, 300, 100):
        t, p = g.gmm_sample(l[i:i + 100], u[i:i + 100], **kw)
        assert torch.equal(t, tokens[i:i + 100]) and torch.equal(p, logp[i:i + 100])
    check(g, l[5:9], u[5:9], unsure=0.25, **kw)


def test_long_rows_captured_and_on_two_streams(g):
    l, u = make((30, 40001), BF16)  # noqa: E741
    step = lambda **kw: g.gmm_sample(l, u, temperature=0.8, top_k=40, top_p=0.9, **kw)  # noqa: E731
    step()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    for k in range(4):
        l.normal_()
        u.uniform_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want)), k
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))


@pytest.mark.parametrize("kw", [dict(temperature=0.0), dict(top_k=1), dict(top_k=7), dict(top_p=0.9), dict(), dict(min_p=0.5)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [301, 40003])
def test_nan_beside_the_largest_value(g, V, dtype, kw):
    """NaN below, above and on both sides of +inf or of float32's largest value, in one piece of 16 bytes and at a row's end."""
    l, u = make((6, V), dtype)  # noqa: E741
    nan, top = float("nan"), math.inf
    l[0, 0], l[0, 1] = nan, top
    l[1, V // 2 // 8 * 8], l[1, V // 2 // 8 * 8 + 3] = nan, torch.finfo(dtype).max
    l[2, 16], l[2, 17], l[2, 18] = nan, top, nan
    l[3, V - 2], l[3, V - 1] = nan, top
    l[4, 8:16], l[4, 15] = nan, top
    l[5, 24:27], l[5, 26:28] = nan, top
    tokens, _ = check(g, l, u, unsure=0.2, **kw)
    if kw.get("temperature") == 0.0 or kw.get("top_k") == 1:
        assert tokens.tolist() == [1, V // 2 // 8 * 8 + 3, 17, V - 1, 15, 26]


@pytest.mark.parametrize("kw", FILTERS)
def test_infinite_logits_among_nan_in_long_rows(g, kw):
    V = 40003
    l, u = make((3, V))  # noqa: E741
    l[:, ::3] = float("nan")
    l[0, 35002] = math.inf
    l[1, 35002:35005] = math.inf
    l[2, 20] = torch.finfo(F32).max
    check(g, l, u, unsure=0.34, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(top_p=0.9), dict(top_p=0.99), dict(top_p=0.5), dict(top_k=40, top_p=0.9), dict(min_p=0.1)])
@pytest.mark.parametrize("V", [300, 20000, 40003])
def test_temperatures_near_the_ends_of_float32(g, V, kw):
    """Logits a few of float32's smallest steps apart under a temperature as small,
    and logits further apart than float32's largest value under one as large."""
    i = torch.arange(V, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(V)
    u = torch.rand(4, generator=gen, device="cuda")
    small = (i * 2000 // V - (1 << 31)).int().view(F32)  # 0 to -1999 steps of 2^-149
    rows = torch.stack([small[torch.randperm(V, generator=gen, device="cuda")] for _ in range(4)])
    tokens, logp = check(g, rows, u, unsure=0.26, temperature=1e-43, **kw)
    many = g.gmm_sample(rows.repeat(75, 1), u.repeat(75), temperature=1e-43, **kw)  # fewer threads a row, more steps each
    assert torch.equal(many[0], tokens.repeat(75)) and torch.equal(many[1], logp.repeat(75))
    large = 6.7e38 * (torch.rand(4, V, generator=gen, device="cuda", dtype=torch.float64) - 0.5)
    check(g, large.float(), u, unsure=0.26, temperature=1e38, **kw)


def test_more_long_rows_than_are_in_flight(g):
    """1040 rows in parts, 1024 at a time over one workspace: each as in a call of its own."""
    R, V = 1040, 32769
    l, u = make((R, V), BF16, pad=5)  # noqa: E741
    i = torch.arange(R, device="cuda")
    kw = dict(temperature=torch.tensor([0.7, 0.0, 1.0, 1.3], device="cuda")[i % 4],
              top_k=torch.tensor([0, 50, 5000], dtype=torch.int32, device="cuda")[i % 3],
              top_p=torch.tensor([0.9, 1.0, 0.999, 0.5, 1.0], device="cuda")[i % 5],
              min_p=torch.tensor([0.0, 0.05], device="cuda")[i % 7 % 2])
    tokens, logp = g.gmm_sample(l, u, **kw)
    for r in [0, 1, 511] + list(range(1020, R)):
        t, p = g.gmm_sample(l[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in kw.items()})
        assert t.item() == tokens[r].item() and p.item() == logp[r].item(), r
    at = torch.tensor([0, 1023, 1024, 1039], device="cuda")
    check(g, l[at], u[at], unsure=0.25, **{k: v[at] for k, v in kw.items()})
