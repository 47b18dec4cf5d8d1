"""GPU parity of expert routing: the sort bit for bit against the oracle's plain
grouping, the moved rows and gradients against float64, and the experts'
products on MXFP4 weights elementwise.

Tolerances: a combined row is a sum of top_k products in fp32 (each product and
addition off by at most 2^-24 relative: (top_k + 1) 2^-23 sum |w ys| covers
both) with one rounding to its type; d_weights is an fp32 sum of d products;
dYs is one fp32 product, rounded again to its type.  The experts' product: as
in the MXFP4 tests."""
import numpy as np
import pytest
import torch

import oracle
import segmented_rank_gemm_segment_amd as srg
import workloads as wl
from gpu_harness import DEV, say
from test_gpu_mxfp4 import U, bf16_device, check_close, mx_device, packed, product_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    srg.lib()
    yield
    torch.cuda.synchronize()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make_ids(seed, n, k, E, kind):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        ids = rng.integers(0, E, size=(n, k))            # repeats within a token occur
    elif kind == "skewed":
        ids = np.minimum((rng.random((n, k)) ** 4 * E).astype(np.int64), E - 1)
    elif kind == "one":
        ids = np.full((n, k), E - 1)
    elif kind == "none":
        ids = np.full((n, k), -1)
    else:                                                # "bad": dropped and invalid ids too
        ids = rng.integers(-4, E + 3, size=(n, k))
        ids[rng.random((n, k)) < 0.02] = 2 ** 31 - 1
        ids[rng.random((n, k)) < 0.02] = -2 ** 31
    return np.ascontiguousarray(ids.astype(np.int32))


def sorted_batch(ids, E):
    n, k = ids.shape
    ex = srg.Experts(n, k, E, DEV)
    ex.sorted_choice.fill_(-7)
    srg.lora_experts_sort(torch.from_numpy(ids).to(DEV), ex)
    return ex


SORTS = [
    (0, 2, 4, "uniform"), (1, 1, 1, "uniform"), (1, 64, 3, "uniform"), (7, 3, 5, "bad"),
    (64, 8, 128, "skewed"), (63, 2, 1024, "uniform"), (512, 2, 1, "one"), (513, 2, 1000, "bad"),
    (1000, 8, 64, "skewed"), (1024, 8, 1024, "bad"), (1025, 8, 33, "uniform"), (3000, 3, 17, "none"),
    (20000, 4, 256, "skewed"), (16384, 8, 1024, "bad"), (50000, 1, 2, "one"),
    (262145, 1, 7, "skewed"), (270000, 1, 1024, "bad"),
]


@pytest.mark.parametrize("n,k,E,kind", SORTS)
def test_sort(n, k, E, kind):
    say("sort", n, k, E, kind)
    ids = make_ids(n + E, n, k, E, kind)
    ex = sorted_batch(ids, E)
    ref = oracle.expert_routing(ids, E)
    kept = len(ref["sorted_choice"])
    assert np.array_equal(ex.expert_offsets.cpu().numpy(), ref["expert_offsets"])
    got = ex.sorted_choice.cpu().numpy()
    assert np.array_equal(got[:kept], ref["sorted_choice"]) and np.all(got[kept:] == -7)
    assert np.array_equal(ex.choice_position.cpu().numpy(), ref["choice_position"])
    assert int(ex.status.item()) == ref["status"]


ROWS = [
    # n, k, E, d, kind
    (1, 1, 1, 8, "uniform"), (1, 4, 8, 136, "uniform"), (5, 3, 4, 24, "bad"), (64, 8, 128, 1032, "skewed"),
    (33, 5, 7, 4096, "bad"), (300, 2, 8, 520, "none"), (4095, 2, 16, 64, "bad"), (4500, 6, 16, 72, "bad"),
    (9, 64, 100, 40, "uniform"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k,E,d,kind", ROWS)
def test_rows_and_gradients(n, k, E, d, kind, dtype):
    say("rows", n, k, E, d, kind, dtype)
    ids = make_ids(n + d, n, k, E, kind)
    ref = oracle.expert_routing(ids, E)
    order, pos = ref["sorted_choice"], ref["choice_position"]
    kept = len(order)
    ex = sorted_batch(ids, E)
    g = torch.Generator(DEV).manual_seed(n)

    def rows(m, fill=None):                              # padded rows: strides are not the width
        t = torch.full((m, d + 8), 5.0, dtype=dtype, device=DEV)
        if fill is None:
            t[:, :d] = torch.randn(m, d, device=DEV, generator=g).to(dtype)
        return t[:, :d]

    X, Ys, dY = rows(n), rows(n * k), rows(n)
    if kept < n * k:
        Ys[kept:] = float("nan")                         # never read
    w = torch.randn(n, k, device=DEV, generator=g)
    Xs, Y, dYs = rows(n * k, 5.0), rows(n, 5.0), rows(n * k, 5.0)
    Y1 = rows(n, 5.0)
    dw = torch.full((n, k), 9.0, device=DEV)
    srg.lora_experts_gather(X, ex, Xs)
    srg.lora_experts_combine(Ys, w, ex, Y)
    srg.lora_experts_combine(Ys, None, ex, Y1)
    srg.lora_experts_combine_backward(dY, Ys, w, ex, dYs, dw)

    f = lambda t: t.double().cpu().numpy()               # noqa: E731
    assert np.array_equal(f(Xs)[:kept], f(X)[order // k])
    for t in (Xs, dYs):
        assert bool((t[kept:] == 5.0).all())
    for t, base in ((Xs, 5.0), (Y, 5.0), (dYs, 5.0)):
        assert bool((t._base[:, d:] == base).all())
    ys = np.where((pos >= 0)[..., None], f(Ys)[np.maximum(pos, 0)], 0.0)
    h = half_step(dtype)
    for out, wt in ((Y, f(w)), (Y1, np.ones((n, k)))):
        want = (wt[..., None] * ys).sum(1)
        tol = h * np.abs(want) * 1.01 + (k + 1) * U * (np.abs(wt[..., None]) * np.abs(ys)).sum(1)
        check_close(out, want, tol, "combine")
    wantw = (ys * f(dY)[:, None]).sum(-1)
    tolw = (d + 2) * U * (np.abs(ys) * np.abs(f(dY))[:, None]).sum(-1)
    check_close(dw, wantw, tolw, "d_weights")
    wantys = f(w).reshape(-1)[order, None] * f(dY)[order // k]
    check_close(dYs[:kept], wantys, (h + 2.0 ** -23) * np.abs(wantys), "dYs")

    # either gradient alone gives the same bits
    d2, w2 = rows(n * k, 5.0), torch.full((n, k), 9.0, device=DEV)
    srg.lora_experts_combine_backward(dY, None, w, ex, d2, None)
    srg.lora_experts_combine_backward(dY, Ys, w, ex, None, w2)
    assert torch.equal(d2, dYs) and torch.equal(w2, dw)


def test_gradients_against_differences():
    """<dY, Y> as a function of the weights and sorted rows is linear in each:
    its difference quotients are the gradients."""
    n, k, E, d = 6, 3, 4, 16
    ids = make_ids(2, n, k, E, "bad")
    ex = sorted_batch(ids, E)
    kept = int(ex.expert_offsets[-1])
    g = torch.Generator(DEV).manual_seed(1)
    # multiples of 1/4 in [-1, 1]: every sum below is exact in fp32
    q = lambda *s: torch.randint(-4, 5, s, device=DEV, generator=g).float() / 4   # noqa: E731
    Ys, w, dY, X, dXs = q(n * k, d), q(n, k), q(n, d), q(n, d), q(n * k, d)
    dYs, dw, Y = torch.zeros(n * k, d, device=DEV), torch.zeros(n, k, device=DEV), torch.zeros(n, d, device=DEV)
    srg.lora_experts_combine_backward(dY, Ys, w, ex, dYs, dw)

    def loss(ys, wt):
        srg.lora_experts_combine(ys, wt, ex, Y)
        return float((Y.double() * dY.double()).sum())

    at = loss(Ys, w)
    for i in range(n):
        for j in range(k):
            w2 = w.clone()
            w2[i, j] += 0.5
            assert (loss(Ys, w2) - at) / 0.5 == float(dw[i, j])
    for p in range(n * k):
        y2 = Ys.clone()
        y2[p, p % d] += 0.5
        want = float(dYs[p, p % d]) if p < kept else 0.0
        assert (loss(y2, w) - at) / 0.5 == want
    # the gather's gradient: combine with weights of one
    dX, Xs = torch.zeros(n, d, device=DEV), torch.zeros(n * k, d, device=DEV)
    srg.lora_experts_combine(dXs, None, ex, dX)

    def gathered(x):
        srg.lora_experts_gather(x, ex, Xs)
        return float((Xs[:kept].double() * dXs[:kept].double()).sum())

    at = gathered(X)
    for i in range(n):
        x2 = X.clone()
        x2[i, i] += 0.5
        assert (gathered(x2) - at) / 0.5 == float(dX[i, i])


PRODUCTS = [
    # n, k, E, d_in, d_out, kind
    (1, 1, 1, 32, 8, "uniform"), (1, 2, 4, 96, 40, "uniform"), (9, 3, 5, 160, 72, "bad"),
    (64, 8, 128, 512, 136, "skewed"), (33, 4, 300, 64, 16, "uniform"), (40, 2, 8, 1056, 264, "bad"),
    (256, 1, 1, 288, 264, "one"), (700, 2, 3, 224, 136, "skewed"), (300, 2, 16, 96, 520, "none"),
    (2500, 4, 6, 160, 264, "bad"), (60, 3, 600, 64, 24, "uniform"),
]


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("n,k,E,d_in,d_out,kind", PRODUCTS)
def test_experts_product(n, k, E, d_in, d_out, kind, gathered):
    say("product", n, k, E, d_in, d_out, kind, gathered)
    ids = make_ids(n + d_in, n, k, E, kind)
    ref = oracle.expert_routing(ids, E)
    order = ref["sorted_choice"]
    kept = len(order)
    ex = sorted_batch(ids, E)
    codes, scales = wl.make_mxfp4(E + d_out, E * d_out, d_in)
    Wq, ws = mx_device(codes, scales)
    Wq = Wq.as_strided((E, d_out, d_in // 2), (d_out * Wq.stride(0), Wq.stride(0), 1))
    ws = ws.as_strided((E, d_out, d_in // 32), (d_out * ws.stride(0), ws.stride(0), 1))
    rows = n if gathered else n * k
    w = wl.make_random(n + 5, rows, d_in, 8, 1, 8, dtype="bf16")
    X = torch.full((rows, d_in + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    X[:, :d_in] = bf16_device(w.X)
    Y = torch.full((n * k, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_experts_gemm_mxfp4w(X[:, :d_in], ex, Wq, ws, Y[:, :d_out], gathered=gathered)
    X64 = oracle.decode(w.X, "bf16")
    off = ref["expert_offsets"]
    for e in range(E):
        if off[e] == off[e + 1]:
            continue
        W64 = oracle.decode_mxfp4(codes[e * d_out:(e + 1) * d_out], scales[e * d_out:(e + 1) * d_out])
        p = np.arange(off[e], off[e + 1])
        Xe = X64[order[p] // k] if gathered else X64[p]
        Y64 = Xe @ W64.T
        d = np.abs(Y[off[e]:off[e + 1], :d_out].double().cpu().numpy() - Y64)
        assert np.all(d <= product_tol(Xe, W64, Y64)), e
    assert bool((Y[kept:] == 7.0).all()) and bool((Y[:, d_out:] == 7.0).all())


@pytest.mark.parametrize("n,k,E,d_in,d_out,kind", [
    (3000, 2, 5, 512, 520, "uniform"), (5000, 4, 9, 1024, 1096, "skewed"), (4100, 2, 3, 1536, 264, "bad"),
    (6000, 3, 12, 128, 2056, "skewed"), (2048, 1, 2, 608, 72, "one")])
def test_experts_product_of_long_segments(n, k, E, d_in, d_out, kind):
    """Segments of many tiles, aligned scale rows; every element."""
    ids = make_ids(n + d_in, n, k, E, kind)
    ref = oracle.expert_routing(ids, E)
    order, off = ref["sorted_choice"], ref["expert_offsets"]
    ex = sorted_batch(ids, E)
    codes, scales = wl.make_mxfp4(E + d_out, E * d_out, d_in)
    Wq, ws = packed(codes, scales)
    Wq = Wq.view(E, d_out, d_in // 2)
    ws = ws.as_strided((E, d_out, d_in // 32), (d_out * ws.stride(0), ws.stride(0), 1))
    X = torch.randn(n, d_in, device=DEV, generator=torch.Generator(DEV).manual_seed(n)).bfloat16()
    Y = torch.full((n * k, d_out), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_experts_gemm_mxfp4w(X, ex, Wq, ws, Y)
    for e in range(E):
        W64 = torch.from_numpy(oracle.decode_mxfp4(codes[e * d_out:(e + 1) * d_out],
                                                   scales[e * d_out:(e + 1) * d_out])).to(DEV)
        X64 = X.double()[torch.from_numpy(order[off[e]:off[e + 1]] // k).long().to(DEV)]
        Y64 = X64 @ W64.t()
        tol = 2.0 ** -8 * Y64.abs() + d_in * U * (X64.abs() @ W64.abs().t())
        assert bool(((Y[off[e]:off[e + 1]].double() - Y64).abs() <= tol).all()), e
    assert bool((Y[len(order):] == 7.0).all())


@pytest.mark.parametrize("n,k,E,d_in,d_out", [
    (400, 2, 20, 256, 2056), (300, 4, 40, 512, 1032), (3000, 2, 5, 64, 2056), (3000, 2, 5, 192, 2056)])
def test_experts_product_on_fresh_operands(n, k, E, d_in, d_out):
    """One to a few stages of K on operands copied right before the call."""
    ids = make_ids(n + d_in, n, k, E, "uniform")
    ref = oracle.expert_routing(ids, E)
    order, off = ref["sorted_choice"], ref["expert_offsets"]
    codes, scales = wl.make_mxfp4(E + d_out, E * d_out, d_in)
    X = torch.randn(n, d_in, generator=torch.Generator().manual_seed(n)).bfloat16()
    W64 = torch.from_numpy(oracle.decode_mxfp4(codes, scales)).to(DEV).view(E, d_out, d_in)
    for rep in range(3):
        ex = sorted_batch(ids, E)
        Wq, ws = packed(codes, scales)
        Wq = Wq.view(E, d_out, d_in // 2)
        ws = ws.as_strided((E, d_out, d_in // 32), (d_out * ws.stride(0), ws.stride(0), 1))
        Xd = X.to(DEV)
        Y = torch.full((n * k, d_out), 7.0, dtype=torch.bfloat16, device=DEV)
        srg.lora_experts_gemm_mxfp4w(Xd, ex, Wq, ws, Y)
        for e in range(E):
            X64 = Xd.double()[torch.from_numpy(order[off[e]:off[e + 1]] // k).long().to(DEV)]
            Y64 = X64 @ W64[e].t()
            tol = 2.0 ** -8 * Y64.abs() + d_in * U * (X64.abs() @ W64[e].abs().t())
            assert bool(((Y[off[e]:off[e + 1]].double() - Y64).abs() <= tol).all()), (rep, e)


@pytest.mark.parametrize("d", [8, 520])
def test_rows_of_more_tokens_than_one_launch(d):
    """2^22 + 3 tokens: rows move in two launches, of one and of four waves a
    token; every row against indexing."""
    n, k, E = (1 << 22) + 3, 1, 3
    g = torch.Generator(DEV).manual_seed(d)
    ids = torch.randint(-1, E, (n, k), device=DEV, generator=g, dtype=torch.int32)
    ex = srg.Experts(n, k, E, DEV)
    srg.lora_experts_sort(ids, ex)
    kept = int(ex.expert_offsets[E])
    rows = torch.argsort(torch.where(ids < 0, E, ids).view(-1), stable=True)[:kept]
    assert torch.equal(ex.sorted_choice[:kept].long(), rows)
    X = torch.randint(-9, 10, (n, d), device=DEV, generator=g, dtype=torch.int8).bfloat16()
    Xs = torch.full((n, d), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_experts_gather(X, ex, Xs)
    assert torch.equal(Xs[:kept], X[rows]) and bool((Xs[kept:] == 7.0).all())
    w = torch.randint(1, 4, (n, k), device=DEV, generator=g).float()
    Y = torch.full((n, d), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_experts_combine(Xs, w, ex, Y)                 # small integers: exact
    wx = torch.where(ids >= 0, w, 0.0)
    assert torch.equal(Y, (X * wx).bfloat16())
    dYs, dw = torch.full_like(Xs, 7.0), torch.full_like(w, 7.0)
    srg.lora_experts_combine_backward(X, Xs, w, ex, dYs, dw)
    assert torch.equal(dYs[:kept], (X * w).bfloat16()[rows]) and bool((dYs[kept:] == 7.0).all())
    assert torch.equal(dw, torch.where(ids >= 0, (X * X).sum(1, keepdim=True, dtype=torch.float32), 0.0))


def test_layer_run_in_a_graph():
    """An expert layer as a model calls it (sort, two products, combine, then the
    combine's gradients), captured once and replayed on new inputs, against the
    same calls made eagerly on another stream and against float64."""
    n, k, E, d, f = 48, 3, 10, 128, 64
    c1, s1 = wl.make_mxfp4(31, E * 2 * f, d, 120, 124)
    c2, s2 = wl.make_mxfp4(32, E * d, f, 120, 124)
    (W1, w1), (W2, w2) = mx_device(c1, s1), mx_device(c2, s2)
    W1, w1 = (t.as_strided((E, 2 * f, t.shape[1]), (2 * f * t.stride(0), t.stride(0), 1)) for t in (W1, w1))
    W2, w2 = (t.as_strided((E, d, t.shape[1]), (d * t.stride(0), t.stride(0), 1)) for t in (W2, w2))

    def buffers():
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)   # noqa: E731
        return dict(ex=srg.Experts(n, k, E, DEV), h=z(n * k, 2 * f), y=z(n * k, d), out=z(n, d),
                    dys=z(n * k, d), dw=z(n, k, t=torch.float32))

    X, dY = (torch.zeros((n, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ids = torch.zeros((n, k), dtype=torch.int32, device=DEV)
    wt = torch.zeros((n, k), device=DEV)

    def step(b):
        srg.lora_experts_sort(ids, b["ex"])
        srg.lora_experts_gemm_mxfp4w(X, b["ex"], W1, w1, b["h"])
        a = (torch.nn.functional.silu(b["h"][:, :f].float()) * b["h"][:, f:].float()).bfloat16()
        srg.lora_experts_gemm_mxfp4w(a, b["ex"], W2, w2, b["y"], gathered=False)
        srg.lora_experts_combine(b["y"], wt, b["ex"], b["out"])
        srg.lora_experts_combine_backward(dY, b["y"], wt, b["ex"], b["dys"], b["dw"])

    b = buffers()
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    side = torch.cuda.Stream()
    for r in range(4):
        host = make_ids(r, n, k, E, "bad")
        ids.copy_(torch.from_numpy(host))
        g = torch.Generator(DEV).manual_seed(r)
        for t in (X, dY, wt):
            t.copy_(torch.randn(t.shape, device=DEV, generator=g))
        for t in ("h", "y", "dys"):
            b[t].zero_()
        graph.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            e = buffers()
            step(e)
        side.synchronize()
        for t in ("h", "y", "out", "dys", "dw"):
            assert torch.equal(b[t], e[t]), t
        ref = oracle.expert_routing(host, E)
        h64 = np.zeros((n * k, 2 * f))
        x64 = X.double().cpu().numpy()
        for p, c in enumerate(ref["sorted_choice"]):
            x = int(host.reshape(-1)[c])
            h64[p] = oracle.decode_mxfp4(c1[x * 2 * f:(x + 1) * 2 * f], s1[x * 2 * f:(x + 1) * 2 * f]) @ x64[c // k]
        got = b["h"].double().cpu().numpy()
        assert np.max(np.abs(got - h64)) <= 2.0 ** -7 * np.max(np.abs(h64))
