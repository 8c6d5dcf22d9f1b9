"""gmm_softmax_xent and gmm_softmax_xent_grad against the plain 64-bit form, on
the GPU: every element of every output inside the bound that its arithmetic
gives (tests/head_ref.py)."""
import numpy as np
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


def make(N, D, V, dtype, bias=True, ignored=0.1, pad=0, offset=0, seed=0, B=None, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 7919 * N + 31 * D + V)
    lead = (N,) if B is None else (B, N)
    X = torch.randn(*lead, D + pad + offset, generator=gen, device="cuda").to(TYPES[dtype])[..., offset:offset + D]
    W = (torch.randn(V, D + offset, generator=gen, device="cuda") * (spread / D ** 0.5)).to(TYPES[dtype])[:, offset:]
    b = torch.randn(V, generator=gen, device="cuda") if bias else None
    y = torch.randint(0, V, lead, generator=gen, device="cuda", dtype=torch.int32)
    y = y.masked_fill(torch.rand(lead, generator=gen, device="cuda") < ignored, -1)
    gl = torch.rand(lead, generator=gen, device="cuda") / N
    return X, W, b, y, gl


def check(g, X, W, b, y, gl, grads=("dX", "dW", "db")):
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    want, tol = ref.xent(X, W, y, b, gl)
    ref.within("lse", lse, want["lse"], tol["lse"])
    ref.within("loss", loss, want["loss"], tol["loss"])
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    assert (db is None) == (b is None)
    for name, got in (("dX", dX), ("dW", dW), ("db", db)):
        if got is not None and name in grads:
            ref.within(name, got, want[name], tol[name])
    return loss, lse, dX, dW, db


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,D,V", [(1, 64, 100), (1, 1, 1), (1, 7, 2), (5, 8, 63), (16, 128, 64), (17, 65, 65), (33, 40, 300),
                                   (64, 256, 1000), (65, 64, 129), (130, 33, 257), (128, 128, 128), (300, 515, 1003),
                                   (777, 130, 501), (1000, 96, 2), (257, 1000, 4100)])
def test_sizes(g, dtype, N, D, V):
    check(g, *make(N, D, V, dtype))


@pytest.mark.parametrize("dtype,N,D,V", [("f32", 300, 1000, 10), ("f32", 129, 700, 517), ("f32", 871, 1300, 77),
                                         ("f32", 70, 400, 1), ("bf16", 130, 2048, 300), ("f16", 200, 4100, 131),
                                         ("f32", 66, 520, 1025), ("bf16", 65, 8192, 513)])
def test_few_tiles_over_long_rows(g, dtype, N, D, V):
    X, W, b, y, gl = make(N, D, V, dtype)
    whole = check(g, X, W, b, y, gl)
    again = check(g, X, W, b, y, gl)
    assert all(torch.equal(p, q) for p, q in zip(whole, again))
    # one of the gradients alone
    _, lse, dX, dW, db = whole
    for i, want in ((0, dict(dW=False, dbias=False)), (1, dict(dX=False, dbias=False))):
        only = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, **want)
        assert torch.equal(only[i], (dX, dW)[i])


@pytest.mark.parametrize("N,D,V,pad,offset,bias", [(65, 129, 2, 0, 0, True), (200, 200, 16, 3, 1, True), (1000, 515, 17, 0, 0, False),
                                                   (777, 1030, 33, 13, 5, True), (3000, 260, 64, 8, 0, True),
                                                   (130, 4099, 64, 0, 2, False), (40, 300, 22, 0, 0, True),
                                                   (500, 300, 65, 0, 0, True), (70, 1000, 128, 1, 0, True), (300, 520, 97, 0, 3, False)])
def test_few_classes_over_wide_float32_rows(g, N, D, V, pad, offset, bias):
    whole = check(g, *make(N, D, V, "f32", pad=pad, offset=offset, bias=bias))
    again = check(g, *make(N, D, V, "f32", pad=pad, offset=offset, bias=bias))
    assert all(p is None and q is None or torch.equal(p, q) for p, q in zip(whole, again))


def test_few_classes_over_problems_apart(g):
    X, W, b, y, gl = make(90, 200, 20, "f32", B=4, pad=5)
    check(g, X, W, b, y, gl)
    check(g, X[:, :41], W, b, y[:, :41].contiguous(), gl[:, :41].contiguous())


def test_few_classes_over_chunks_of_rows(g):
    check(g, *make((1 << 20) + 77, 130, 5, "f32", ignored=0.02))


@pytest.mark.parametrize("N,D,V", [(70, 1500, 600), (400, 1500, 600), (150, 300, 40)])
def test_few_tiles_with_masked_classes_and_rows(g, N, D, V):
    X, W, b, y, gl = make(N, D, V, "f32", ignored=0.4)
    b[3 : V - 10] = -float("inf")  # a span without a class
    y.copy_(torch.where(y < 0, y, y % 3))
    X[y < 0] = float("nan")
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    assert not loss[y < 0].any() and not dX[y < 0].any()
    assert all(torch.isfinite(t).all() for t in (loss, dX, dW, db)) and not dW[3 : V - 10].any() and not db[3 : V - 10].any()
    y[5] = V
    assert torch.isnan(g.gmm_softmax_xent(X, W, y, bias=b)[0][5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 200])
@pytest.mark.parametrize("pad,offset", [(8, 0), (13, 0), (0, 1), (5, 3), (0, 8)])
def test_strides_and_alignment(g, dtype, N, pad, offset):
    check(g, *make(N, 72, 130, dtype, pad=pad, offset=offset))
    check(g, *make(N, 71, 130, dtype, pad=pad, offset=offset, bias=False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_batched_rows(g, dtype):
    for N, pad in ((40, 0), (40, 8), (9, 3)):
        X, W, b, y, gl = make(N, 64, 90, dtype, B=5, pad=pad)
        whole = check(g, X, W, b, y, gl)
        half_of = X[:, : N // 2]  # problems apart
        part = check(g, half_of, W, b, y[:, : N // 2].contiguous(), gl[:, : N // 2].contiguous())
        assert torch.equal(part[0], whole[0][:, : N // 2]) or N // 2 * 5 <= 64 < N * 5


@pytest.mark.parametrize("dtype,N,D,V", [("bf16", 40000, 8, 5000), ("bf16", 5000, 8, 40000), ("f32", 20000, 16, 5000),
                                         ("f16", 33000, 8, 33000), ("bf16", 4100, 72, 4500), ("f32", 4100, 40, 4500),
                                         ("bf16", 100000, 130, 40)])
def test_chunks_of_rows_and_pieces_of_the_head(g, dtype, N, D, V):
    check(g, *make(N, D, V, dtype, ignored=0.02))


@pytest.mark.parametrize("dtype,N,V", [("f16", 1000, 20000), ("bf16", 1025, 16385), ("f32", 300, 33001)])
def test_classes_past_the_last_whole_round_of_tiles(g, dtype, N, V):
    X, W, b, y, gl = make(N, 136, V, dtype, ignored=0.0)
    y[::3] = V - 1 - torch.arange(len(y[::3]), device="cuda", dtype=torch.int32) % 200  # labels on both sides
    check(g, X, W, b, y, gl)


@pytest.mark.parametrize("N", [7, 200])
def test_rows_left_out_take_no_part(g, N):
    X, W, b, y, gl = make(N, 64, 300, "bf16", ignored=0.5)
    y[0], y[1] = -1, 5
    loss, lse, dX, dW, db = check(g, X, W, b, y, gl)
    X2 = X.clone()
    X2[y < 0] = float("nan")
    gl2 = gl.masked_fill(y < 0, float("inf"))
    loss2, lse2 = g.gmm_softmax_xent(X2, W, y, bias=b)
    dX2, dW2, db2 = g.gmm_softmax_xent_grad(X2, W, y, lse2, gloss=gl2, bias=b)
    assert torch.equal(loss, loss2) and torch.equal(dX, dX2) and torch.equal(dW, dW2) and torch.equal(db, db2)
    assert (loss[y < 0] == 0).all() and (dX[y < 0] == 0).all() and torch.isnan(lse2[y < 0]).all()
    y[:] = -100
    loss, lse = g.gmm_softmax_xent(X2, W, y, bias=b)
    dX, dW, db = g.gmm_softmax_xent_grad(X2, W, y, lse, bias=b)
    assert not loss.any() and not dX.any() and not dW.any() and not db.any()


@pytest.mark.parametrize("N", [4, 150])
def test_label_past_the_head_is_nan(g, N):
    X, W, b, y, gl = make(N, 32, 70, "f32", ignored=0.0)
    y[2] = 70
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    assert torch.isnan(loss[2]) and torch.isnan(loss).sum() == 1 and not torch.isnan(lse).any()
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    assert torch.isnan(dX[2]).all() and torch.isnan(dX).any(dim=1).sum() == 1
    assert torch.isnan(dW).all() and torch.isnan(db).all()


@pytest.mark.parametrize("N", [6, 140])
def test_classes_masked_by_the_bias(g, N):
    X, W, b, y, gl = make(N, 64, 400, "bf16", ignored=0.0)
    b[3:390] = -float("inf")  # whole tiles without a class
    y.copy_(torch.arange(N, device="cuda", dtype=torch.int32) % 3)
    loss, lse, dX, dW, db = check(g, X, W, b, y, gl)
    assert not dW[3:390].any() and not db[3:390].any()
    b[:] = -float("inf")
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    assert (lse == -float("inf")).all() and torch.isnan(loss).all()


@pytest.mark.parametrize("N", [6, 140])
def test_infinite_and_nan_logits(g, N):
    X, W, b, y, gl = make(N, 16, 200, "f32", ignored=0.0)
    X[1, 3] = float("nan")
    X[2, 0] = float("inf")
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[1] = rest[2] = False
    assert torch.isnan(lse[1]) and torch.isnan(lse[2])
    assert torch.isfinite(lse[rest]).all() and torch.isfinite(loss[rest]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_confident_rows_and_large_logits(g, dtype):
    X, W, b, y, gl = make(200, 64, 300, dtype, spread=60.0)
    check(g, X, W, b, y, gl)
    top = (X.float() @ W.float().t() + b).argmax(1).int()
    check(g, X, W, b, top, gl)


def test_row_gradients_of_mixed_size_in_half(g):
    X, W, b, y, gl = make(300, 64, 500, "f16", ignored=0.0)
    gl = torch.exp(torch.linspace(-20, 6, 300, device="cuda"))
    check(g, X, W, b, y, gl)
    check(g, X, W, b, y, torch.zeros_like(gl))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accumulate_and_parts(g, dtype):
    X, W, b, y, gl = make(150, 72, 333, dtype)
    _, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        got = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, **{k: None if on else False for k, on in zip(("dX", "dW", "dbias"), keep)})
        for a, whole, on in zip(got, (dX, dW, db), keep):
            assert (a is None) if not on else torch.equal(a, whole)
    # added once, to what is there: one rounding of the exact sum
    old = [torch.randn_like(t) for t in (dX, dW, db)]
    acc = [t.clone() for t in old]
    g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, dX=acc[0], dW=acc[1], dbias=acc[2], accumulate=True)
    want, tol = ref.xent(X, W, y, b, gl)
    for name, o, a in zip(("dX", "dW", "db"), old, acc):
        s = want[name] + o.double()
        ref.within(name, a, s, tol[name] + (ref.half(a.dtype) + 2 * ref.U) * (s.abs() + o.double().abs() + tol[name]))


def test_no_rows(g):
    X = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    W = torch.randn(100, 64, device="cuda").bfloat16()
    y = torch.empty(0, device="cuda", dtype=torch.int32)
    b = torch.zeros(100, device="cuda")
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    assert loss.shape == (0,) and lse.shape == (0,)
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, bias=b)
    assert dX.shape == (0, 64) and not dW.any() and not db.any()
    acc = torch.ones_like(dW)
    g.gmm_softmax_xent_grad(X, W, y, lse, dX=False, dW=acc, accumulate=True, dbias=False)
    assert (acc == 1).all()


def test_gradient_against_differences(g):
    """Central differences of the 64-bit loss: their own error is h^2 / 6 times
    the third derivative, at most 6 sum_i |g_i| (max |w_v| or |x_i|)^3."""
    X, W, b, y, gl = make(4, 5, 7, "f32", ignored=0.0)
    _, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    _, tol = ref.xent(X, W, y, b, gl)
    x, w, bb, yy, gg = (t.cpu().double().numpy() for t in (X, W, b, y, gl))
    yy = yy.astype(int)

    def f(x, w, bb):
        L = x @ w.T + bb
        m = L.max(1, keepdims=True)
        return float((gg * (m[:, 0] + np.log(np.exp(L - m).sum(1)) - L[np.arange(4), yy])).sum())

    h = 1e-4
    M = max(np.abs(x).max(), np.abs(w).max(), 1.0)
    slack = h * h * np.abs(gg).sum() * (5 * M) ** 3 + 1e-15 / h * 100
    for name, arr, got in (("x", x, dX), ("w", w, dW), ("b", bb, db)):
        diff = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            args = {"x": x, "w": w, "bb": bb}
            key = "bb" if name == "b" else name
            diff[i] = (f(**{**args, key: up}) - f(**{**args, key: dn})) / (2 * h)
        bound = tol[{"x": "dX", "w": "dW", "b": "db"}[name]] + slack
        ref.within("d" + name, got, torch.from_numpy(diff).cuda(), bound)


@pytest.mark.parametrize("N", [10, 500])
def test_same_inputs_same_bits_also_captured_and_on_another_stream(g, N):
    X, W, b, y, gl = make(N, 128, 700, "bf16")

    def step():
        loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
        return (loss, lse) + g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)

    first = [t.clone() for t in step()]
    for a, c in zip(first, step()):
        assert torch.equal(a, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        X.normal_()
        X.mul_(k + 1)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs, step()):
            assert torch.equal(a, c), k
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b, stream=side)
    side.synchronize()
    assert torch.equal(loss, outs[0])


@pytest.mark.parametrize("dtype,N,D,V", [("f32", 500, 300, 20), ("f32", 200, 900, 300), ("bf16", 150, 4096, 200)])
def test_logits_in_parts_captured_and_in_two_streams_at_once(g, dtype, N, D, V):
    X, W, b, y, gl = make(N, D, V, dtype)

    def step():
        loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
        return (loss, lse) + g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)

    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        X.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), k
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for _ in range(3):
        for st in sides:
            with torch.cuda.stream(st):
                got.append(step())
    torch.cuda.synchronize()
    for t in got:
        assert all(torch.equal(p, q) for p, q in zip(t, want))


def test_wide_rows_of_few_classes_far_apart(g):
    """Row offsets past 2^31 bytes."""
    ld = (1 << 22) + 4
    big = torch.empty(300, ld, device="cuda")
    X = big[:, 3:203]
    X.copy_(torch.randn(300, 200, device="cuda"))
    _, W, b, y, gl = make(300, 200, 12, "f32")
    check(g, X, W, b, y, gl)


def test_rows_far_apart(g):
    """Row offsets past 2^31 bytes: rows of a wide array."""
    ld = (1 << 22) + 8
    big = torch.empty(520, ld, device="cuda", dtype=torch.bfloat16)
    X = big[:, :40]
    X.copy_(torch.randn(520, 40, device="cuda"))
    _, W, b, y, gl = make(520, 40, 120, "bf16")
    check(g, X, W, b, y, gl)
    check(g, X[::40], W, b, y[::40].contiguous(), gl[::40].contiguous())


LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,D,V", [(6, 64, 300), (140, 64, 300), (140, 20, 3000), (140, 128, 77), (140, 200, 300), (20000, 40, 500)])
def test_every_class_masked_with_the_lowest_value(g, dtype, N, D, V):
    """float32 has no room for log V beside 3.4e38: lse is the mask's value, on
    every path, and what follows from it is finite."""
    X, W, b, y, gl = make(N, D, V, dtype, ignored=0.0)
    b[:] = LOWEST
    loss, lse, dX, dW, db = check(g, X, W, b, y, gl)
    assert torch.equal(lse, torch.full_like(lse, LOWEST)) and torch.isfinite(loss).all()
    assert all(torch.isfinite(t).all() for t in (dX, dW, db))


@pytest.mark.parametrize("N", [6, 140])
def test_classes_masked_with_the_lowest_value(g, N):
    X, W, b, y, gl = make(N, 64, 400, "bf16", ignored=0.0)
    b[3:390] = LOWEST
    y.copy_(torch.arange(N, device="cuda", dtype=torch.int32) % 3)
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    assert not dW[3:390].any() and not db[3:390].any()
    assert torch.isfinite(loss).all() and torch.isfinite(dX).all()
    b[3:390] = -float("inf")
    again = g.gmm_softmax_xent(X, W, y, bias=b)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,D,V", [(6, 64, 300), (140, 64, 300), (300, 20, 3000), (140, 128, 77), (140, 200, 300), (300, 1000, 100)])
def test_one_class_far_above_the_rest(g, dtype, N, D, V):
    """A logit of 3e38, whose product with log2(e) leaves float32: p is 1 there
    and 0 elsewhere, so G is g ([v = 7] - [v = y]) without any error of its own;
    what is left is G's rounding to the rows' type (half a step), the sums and
    the last rounding."""
    X, W, b, y, gl = make(N, D, V, dtype, ignored=0.0)
    b[7] = 3e38
    y[::2] = 7
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    assert (lse == b[7]).all() and not loss[::2].any()
    dX, dW, db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    G = torch.zeros(N, V, dtype=torch.float64, device="cuda")
    G[:, 7] = gl.double()
    G[torch.arange(N, device="cuda"), y.long()] -= gl.double()
    h = ref.half(X.dtype)
    for name, got, a, c in (("dX", dX, G, W.double()), ("dW", dW, G.t().contiguous(), X.double())):
        want, mag = a @ c, a.abs() @ c.abs()
        tol = (h + (V + N + 8) * ref.U) * mag
        ref.within(name, got, want, tol + (h + 2 * ref.U) * (want.abs() + tol) + ref.tiny(X.dtype))
    ref.within("db", db, G.sum(0), (N + 8) * ref.U * G.abs().sum(0))


@pytest.mark.parametrize("dtype,N,D,V", [("f16", 34000, 130, 33000), ("bf16", 60000, 136, 5000), ("f32", (3 << 20) + 5, 24, 40)])
def test_bias_gradient_over_chunks_of_rows_is_added_once(g, dtype, N, D, V):
    """Whatever the chunks: the sum, inside its own bound, and one rounding of
    what it is added to."""
    X, W, b, y, gl = make(N, D, V, dtype, ignored=0.02)
    _, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    want, tol = ref.xent(X, W, y, b, gl)
    only = dict(dX=False, dW=False)
    db = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, **only)[2]
    ref.within("db", db, want["db"], tol["db"])
    old = torch.randn(V, device="cuda") * 100
    acc = old.clone()
    g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, dbias=acc, accumulate=True, **only)
    s = old.double() + want["db"]
    ref.within("db", acc, s, tol["db"] + 1.01 * ref.U * (s.abs() + tol["db"]))
    assert torch.equal(acc, old + db)


def in_pieces(g, N, D, V, dtype):
    """Whether a gradient call forms G in pieces: its workspace for the bias
    gradient alone, which is one piece and little else, is below all of G."""
    import ctypes

    from soft_clustering_em_amd import _abi
    code = {"f32": _abi.DT_F32, "bf16": _abi.DT_BF16, "f16": _abi.DT_F16}[dtype]
    d = _abi.GmmData(ctypes.c_void_p(256), code, 1, N, D, D, N * D)
    h = _abi.GmmHead(ctypes.c_void_p(1 << 40), code, V, D, None)
    n = _abi.lib().gmm_softmax_xent_grad_workspace_bytes(ctypes.byref(d), ctypes.byref(h), 4)
    return 0 < n < N * V * (6 if dtype == "f32" else 2)


@pytest.mark.parametrize("dtype,N,D,V", [
    ("bf16", 40000, 136, 5000), ("f32", 20000, 136, 4500),    # chunks of rows
    ("bf16", 5000, 136, 40000), ("f32", 4500, 130, 20000),    # pieces of the classes
    ("bf16", 33000, 136, 33000), ("f32", 33000, 136, 33300),  # both, classes in the outer loop
    ("f16", 34000, 130, 33000), ("f32", 33500, 136, 33000),   # both, rows in the outer loop
    ("f16", 33000, 131, 34000)])
def test_wide_rows_in_chunks_and_classes_in_pieces(g, dtype, N, D, V):
    """Rows and head past what one piece of G holds, the last chunk and piece
    shorter than the others, written and added."""
    assert in_pieces(g, N, D, V, dtype)
    X, W, b, y, gl = make(N, D, V, dtype, ignored=0.02)
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    want, tol = ref.xent(X, W, y, b, gl)
    ref.within("lse", lse, want["lse"], tol["lse"])
    ref.within("loss", loss, want["loss"], tol["loss"])
    got = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b)
    for name, t in zip(("dX", "dW", "db"), got):
        ref.within(name, t, want[name], tol[name])
    old = [torch.randn_like(t) for t in got]
    acc = [t.clone() for t in old]
    g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, dX=acc[0], dW=acc[1], dbias=acc[2], accumulate=True)
    for name, o, a in zip(("dX", "dW", "db"), old, acc):
        s = want[name] + o.double()
        ref.within(name, a, s, tol[name] + (ref.half(a.dtype) + 2 * ref.U) * (s.abs() + o.double().abs() + tol[name]))
    # one of the gradients alone
    for i, only in ((0, dict(dW=False, dbias=False)), (1, dict(dX=False, dbias=False)), (2, dict(dX=False, dW=False))):
        assert torch.equal(g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, **only)[i], got[i])


@pytest.mark.parametrize("dtype,N,D,V", [("bf16", 22000, 136, 100000), ("f32", 22000, 130, 100000)])
def test_loss_of_wide_rows_in_chunks(g, dtype, N, D, V):
    """More than 2^24 (maximum, sum) pairs: the loss takes the rows in chunks."""
    assert (V + 127) // 128 * N > 1 << 24
    X, W, b, y, gl = make(N, D, V, dtype, ignored=0.02)
    loss, lse = g.gmm_softmax_xent(X, W, y, bias=b)
    want, tol = ref.xent(X, W, y, b, gl, rows=1 << 11)
    ref.within("lse", lse, want["lse"], tol["lse"])
    ref.within("loss", loss, want["loss"], tol["loss"])


@pytest.mark.parametrize("dtype,N,D,V,offset", [("f32", (1 << 20) + 77, 24, 30, 0), ("bf16", (1 << 20) + 77, 33, 12, 1),
                                                ("f32", 200, 24, (1 << 18) + 100, 0), ("f16", 130, 33, (1 << 18) + 100, 1)])
def test_narrow_rows_and_classes_copied_in_chunks(g, dtype, N, D, V, offset):
    """Rows past 2^20 and classes past 2^18 that are copied to aligned ones first."""
    check(g, *make(N, D, V, dtype, ignored=0.02, offset=offset))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,V", [(5, 130), (70, 130), (300, 700)])
def test_widest_rows(g, dtype, N, V):
    check(g, *make(N, 65536, V, dtype))


@pytest.mark.parametrize("D", [136, 64])
def test_rows_and_classes_as_far_apart_as_loads_reach(g, D):
    """256 rows just inside 2^31 bytes: taken where they lie."""
    ld = 4194296
    big = torch.empty(300, ld, device="cuda", dtype=torch.bfloat16)
    X, W, b, y, gl = make(300, D, 300, "bf16")
    for far, other in ((X, W), (W, X)):
        at = big[:, :D]
        at.copy_(far)
        check(g, *((at, other) if far is X else (other, at)), b, y, gl)


def test_problems_of_one_row(g):
    check(g, *make(1, 40, 30, "f32", B=70000))
    check(g, *make(1, 200, 30, "bf16", B=7000, pad=8))


@pytest.mark.parametrize("N,D", [(20, 64), (200, 64), (200, 300)])
def test_labels_at_the_ends_of_their_type(g, N, D):
    X, W, b, y, gl = make(N, D, 100, "bf16", ignored=0.0)
    y[3], y[7] = -(2 ** 31), 5 - 2 ** 31
    check(g, X, W, b, y, gl)
    y[5] = 2 ** 31 - 1
    loss, _ = g.gmm_softmax_xent(X, W, y, bias=b)
    assert torch.isnan(loss[5]) and torch.isnan(loss).sum() == 1


def test_captured_with_its_stream_named(g):
    X, W, b, y, gl = make(300, 64, 100, "bf16")
    want = g.gmm_softmax_xent(X, W, y, bias=b)
    grads = g.gmm_softmax_xent_grad(X, W, y, want[1], gloss=gl, bias=b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss, lse = g.gmm_softmax_xent(X, W, y, bias=b, stream=side)
        outs = g.gmm_softmax_xent_grad(X, W, y, lse, gloss=gl, bias=b, stream=side)
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and all(torch.equal(p, q) for p, q in zip(outs, grads))


def test_more_than_2_27_rows(g):
    """Row numbers past 27 bits, against a sample of the rows."""
    N, D, V = (1 << 27) + 3, 8, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(N, D, generator=gen, device="cuda").bfloat16()
    W = torch.randn(V, D, generator=gen, device="cuda").bfloat16()
    y = torch.randint(-1, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    loss, lse = g.gmm_softmax_xent(X, W, y)
    dX, dW, _ = g.gmm_softmax_xent_grad(X, W, y, lse)
    at = torch.cat([torch.arange(0, N, 9973, device="cuda"), torch.arange(N - 1000, N, device="cuda")])
    want, tol = ref.xent(X[at].contiguous(), W, y[at].contiguous())
    for name, t in (("lse", lse), ("loss", loss), ("dX", dX)):
        ref.within(name, t[at], want[name], tol[name])
    # one more than the rows before the last, whose gradient is one row's
    again = g.gmm_softmax_xent_grad(X[:-1], W, y[:-1], lse[:-1], dX=False)[1]
    assert torch.isfinite(dW).all() and float((dW.double() - again.double()).abs().max()) <= 2 * ref.half(X.dtype) * float(dW.double().abs().max())
