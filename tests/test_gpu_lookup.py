"""gmm_codebook_lookup and gmm_codebook_lookup_grad against the plain 64-bit
form, on the GPU, element by element (bounds: tests/head_ref.py)."""
import pytest
import torch

import head_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import soft_clustering_em_amd as g
    return g


def make(N, m, D, K, dtype, weighted=True, seed=0, skew=False, offset=0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 101 * N + 7 * m + 3 * D + K)
    dt = TYPES[dtype]
    table = torch.randn(K, D + offset + pad, generator=gen, device="cuda").to(dt)[:, offset:offset + D]
    dout = torch.randn(N, D + offset + pad, generator=gen, device="cuda").to(dt)[:, offset:offset + D]
    u = torch.rand(N, m, generator=gen, device="cuda")
    idx = (u * u * u * K if skew else u * K).int().clamp_(0, K - 1)
    keep = torch.randint(0, m + 1, (N, 1), generator=gen, device="cuda")
    idx = torch.where(torch.arange(m, device="cuda") < keep, idx, torch.full_like(idx, -1))
    bad = torch.rand(N, m, generator=gen, device="cuda") < 0.05
    idx = torch.where(bad, torch.full_like(idx, K), idx).int().contiguous()
    w = torch.randn(N, m, generator=gen, device="cuda") if weighted else None
    return table, dout, idx, w


SIZES = [(1, 1, 1, 1), (1, 1, 4096, 50), (1, 4, 128, 10), (3, 2, 7, 1), (100, 4, 128, 64), (257, 3, 65, 5), (1000, 1, 33, 2000),
         (4096, 4, 128, 300), (4097, 16, 20, 1000), (5000, 1, 520, 7), (9000, 5, 8, 1030), (70, 1, 8200, 40),
         (30000, 2, 16, 120000), (8192, 1, 12, 700), (2731, 3, 40, 90), (8193, 1, 12, 700), (33, 1, 5, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,m,D,K", SIZES)
def test_lookup(g, dtype, N, m, D, K):
    table, _, idx, w = make(N, m, D, K, dtype)
    for weights, scale in ((w, 1.0), (None, 0.37), (w, -2.5)):
        got = g.gmm_codebook_lookup(table, idx, weights=weights, scale=scale)
        ref.within("rows", got, *ref.lookup(table, idx, weights, float(torch.tensor(scale, dtype=torch.float32))))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,m,D,K", SIZES)
@pytest.mark.parametrize("skew", [False, True])
def test_gradients(g, dtype, N, m, D, K, skew):
    table, dout, idx, w = make(N, m, D, K, dtype, skew=skew)
    for weights, scale in ((w, 1.0), (None, 0.37)):
        s32 = float(torch.tensor(scale, dtype=torch.float32))
        dt, dw = g.gmm_codebook_lookup_grad(dout, idx, K, table=table, weights=weights, scale=scale)
        (want, tol), wdw = ref.lookup_grad(dout, idx, K, table, weights, s32)
        ref.within("dtable", dt, want, tol)
        assert (dw is None) == (weights is None)
        if dw is not None:
            ref.within("dweights", dw, *wdw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(g, dtype, pad, offset):
    for D in (72, 71):
        table, dout, idx, w = make(500, 3, D, 90, dtype, pad=pad, offset=offset)
        ref.within("rows", g.gmm_codebook_lookup(table, idx, weights=w), *ref.lookup(table, idx, w))
        dt, dw = g.gmm_codebook_lookup_grad(dout, idx, 90, table=table, weights=w)
        (want, tol), wdw = ref.lookup_grad(dout, idx, 90, table, w)
        ref.within("dtable", dt, want, tol)
        ref.within("dweights", dw, *wdw)


@pytest.mark.parametrize("N,K", [(100000, 1), (100000, 3), (65537, 2), (40000, 40000)])
def test_codes_with_most_of_the_entries(g, N, K):
    table, dout, idx, w = make(N, 1, 24, K, "f32", skew=True)
    idx[: N // 2] = K - 1
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, K, table=table, weights=w)
    (want, tol), wdw = ref.lookup_grad(dout, idx, K, table, w)
    ref.within("dtable", dt, want, tol)
    ref.within("dweights", dw, *wdw)


def test_no_entries(g):
    table, dout, idx, w = make(50, 3, 40, 20, "bf16")
    idx[:] = -1
    assert not g.gmm_codebook_lookup(table, idx, weights=w).any()
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, 20, table=table, weights=w)
    assert not dt.any() and not dw.any()
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    assert g.gmm_codebook_lookup(table, none).shape == (0, 40)
    dt, _ = g.gmm_codebook_lookup_grad(dout[:0], none, 20)
    assert dt.shape == (20, 40) and not dt.any()


def test_rows_that_end_early_ignore_what_is_behind(g):
    table, dout, idx, w = make(400, 4, 32, 50, "f32")
    w2 = torch.where(ref.entries(idx, 50), w, torch.full_like(w, float("nan")))
    assert torch.equal(g.gmm_codebook_lookup(table, idx, weights=w), g.gmm_codebook_lookup(table, idx, weights=w2))
    a = g.gmm_codebook_lookup_grad(dout, idx, 50, table=table, weights=w)
    b = g.gmm_codebook_lookup_grad(dout, idx, 50, table=table, weights=w2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dead = ~ref.entries(idx, 50).any(1)
    d2 = dout.masked_fill(dead[:, None], float("nan"))
    assert torch.equal(a[0], g.gmm_codebook_lookup_grad(d2, idx, 50, table=table, weights=w)[0])


def test_the_same_code_twice_in_a_row(g):
    table, dout, _, _ = make(300, 2, 40, 10, "f32")
    idx = torch.randint(0, 10, (300, 1), device="cuda", dtype=torch.int32).repeat(1, 2).contiguous()
    ref.within("rows", g.gmm_codebook_lookup(table, idx), *ref.lookup(table, idx))
    (want, tol), _ = ref.lookup_grad(dout, idx, 10)
    ref.within("dtable", g.gmm_codebook_lookup_grad(dout, idx, 10)[0], want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_batched_tables(g, dtype):
    B, N, m, K, D = 3, 210, 3, 33, 40
    parts = [make(N, m, D, K, dtype, seed=b) for b in range(B)]
    table, dout, idx, w = (torch.stack([p[i] for p in parts]) for i in range(4))
    wide = torch.randn(B, K + 5, D + 8, device="cuda").to(table.dtype)
    wide[:, :K, :D] = table
    view = wide[:, :K, :D]
    rows = g.gmm_codebook_lookup(view, idx, weights=w, scale=0.5)
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, K, table=view, weights=w, scale=0.5)
    for b in range(B):
        ref.within("rows", rows[b], *ref.lookup(table[b], idx[b], w[b], 0.5))
        (want, tol), wdw = ref.lookup_grad(dout[b], idx[b], K, table[b], w[b], 0.5)
        ref.within("dtable", dt[b], want, tol)
        ref.within("dweights", dw[b], *wdw)


def test_labels_without_a_slot_axis(g):
    table, dout, idx, _ = make(333, 1, 48, 20, "bf16")
    flat = idx[:, 0].contiguous()
    assert torch.equal(g.gmm_codebook_lookup(table, flat), g.gmm_codebook_lookup(table, idx))
    assert torch.equal(g.gmm_codebook_lookup_grad(dout, flat, 20)[0], g.gmm_codebook_lookup_grad(dout, idx, 20)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_accumulate(g, dtype):
    table, dout, idx, w = make(3000, 2, 40, 64, dtype, skew=True)
    old = torch.randn(64, 40, device="cuda").to(dout.dtype)
    acc = old.clone()
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, 64, weights=w, dtable=acc, accumulate=True)
    assert dt is acc and dw is None
    (want, tol), _ = ref.lookup_grad(dout, idx, 64, None, w, old=old)
    ref.within("dtable", acc, want, tol)
    none = g.gmm_codebook_lookup_grad(dout, idx, 64, table=table, weights=w, dtable=False)
    assert none[0] is None and none[1].shape == idx.shape


def test_gradient_against_differences(g):
    """The lookup is linear: differences of <dout, rows> are exact up to rounding."""
    table, dout, idx, w = make(6, 3, 4, 5, "f32")
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, 5, table=table, weights=w, scale=0.5)
    f = lambda t, ww: float((dout.double() * ref.lookup(t.double(), idx, ww.double(), 0.5)[0]).sum())  # noqa: E731
    (_, tol), (_, wtol) = ref.lookup_grad(dout, idx, 5, table, w, 0.5)
    for got, arr, bound, call in ((dt, table, tol, lambda a: f(a, w)), (dw, w, wtol, lambda a: f(table, a))):
        diff = torch.zeros(arr.shape, dtype=torch.float64, device="cuda")
        for i in range(arr.numel()):
            up, dn = arr.double().clone(), arr.double().clone()
            up.view(-1)[i] += 0.5
            dn.view(-1)[i] -= 0.5
            diff.view(-1)[i] = call(up) - call(dn)
        ref.within("differences", got, diff, bound + 1e-12)


def test_same_inputs_same_bits_also_captured(g):
    table, dout, idx, w = make(20000, 3, 40, 700, "bf16", skew=True)

    def step():
        rows = g.gmm_codebook_lookup(table, idx, weights=w)
        return (rows,) + g.gmm_codebook_lookup_grad(dout, idx, 700, table=table, weights=w)

    first = [t.clone() for t in step()]
    for a, c in zip(first, step()):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        dout.normal_()
        idx.copy_(idx[torch.randperm(20000, device="cuda")])
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs, step()):
            assert torch.equal(a, c), k


def test_table_past_32_bits(g):
    """Offsets past 2^31 elements of a table."""
    K, D = 270000, 8192
    table = torch.zeros(K, D, device="cuda", dtype=torch.bfloat16)
    at = torch.tensor([0, K - 1, K // 2, 262144, 262143], device="cuda")
    table[at] = torch.randn(5, D, device="cuda").bfloat16()
    idx = at.int()
    assert torch.equal(g.gmm_codebook_lookup(table, idx), table[at])
    dout = torch.randn(5, D, device="cuda").bfloat16()
    dt, _ = g.gmm_codebook_lookup_grad(dout, idx, K)
    assert torch.equal(dt[at], dout)
    dt[at] = 0
    assert not dt.any()


@pytest.mark.parametrize("N,m,D,K", [(1, 4096, 8, 50), (40, 700, 20, 90), (7, 17, 33, 5), (600, 33, 12, 3000)])
def test_long_rows(g, N, m, D, K):
    table, dout, idx, w = make(N, m, D, K, "f32")
    gen = torch.Generator(device="cuda").manual_seed(N + m)
    idx = torch.randint(0, K, (N, m), generator=gen, device="cuda", dtype=torch.int32)
    ends = torch.randint(0, m + 1, (N,), generator=gen, device="cuda").tolist()
    for i, e in enumerate(ends):  # one value outside: what is behind it takes no part
        if e < m and N > 1:
            idx[i, e] = (-1, K)[i % 2]
    got = g.gmm_codebook_lookup(table, idx, weights=w)
    ref.within("rows", got, *ref.lookup(table, idx, w, 1.0))
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, K, table=table, weights=w)
    (want, tol), wdw = ref.lookup_grad(dout, idx, K, table, w, 1.0)
    ref.within("dtable", dt, want, tol)
    ref.within("dweights", dw, *wdw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_widest_rows(g, dtype):
    table, dout, idx, w = make(40, 3, 65536, 20, dtype)
    ref.within("rows", g.gmm_codebook_lookup(table, idx, weights=w), *ref.lookup(table, idx, w))
    dt, dw = g.gmm_codebook_lookup_grad(dout, idx, 20, table=table, weights=w)
    (want, tol), wdw = ref.lookup_grad(dout, idx, 20, table, w)
    ref.within("dtable", dt, want, tol)
    ref.within("dweights", dw, *wdw)
