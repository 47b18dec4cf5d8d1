"""Every kernel that the products with MXFP4 operands choose from, reached by its
own shapes (test_mx_choice_cpu.py holds them against the rules), every element
against float64.

Tolerance of an element: its own rounding to bf16, 2^-8 |y|, plus the fp32
accumulation: a sum of K exact products, in any order and grouping, each addition
off by at most 2^-23 of the partial sum, is off by at most K 2^-23 sum |x_c w_c|;
1.01 for the rounding of a result that is off by that.  The LoRA term adds H's sum
over d_in, its own sum over r, the scale's product and the split of s H into two
bf16 parts (2^-16 relative); the base sum and the term meet in one addition a rank
step.  A DoRA factor scales all of that and adds one fp32 product."""
import numpy as np
import pytest
import torch

import oracle
import segmented_rank_gemm_segment_amd as srg
import workloads as wl
from gpu_harness import DEV, say
from test_gpu_mxfp4 import U, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    srg.lib()
    yield
    torch.cuda.synchronize()


def random_rows(n, d, seed):
    return torch.randn(n, d, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)).bfloat16()


def values(codes, scales):
    return torch.from_numpy(oracle.decode_mxfp4(codes, scales)).to(DEV)


def check(out, Y64, acc, what):
    d = (out.double() - Y64).abs()
    tol = 2.0 ** -8 * Y64.abs() + 1.01 * acc
    say(what, "worst error / tolerance", float((d / tol.clamp_min(1e-300)).max()))
    assert bool((d <= tol).all()), what


# n, d_in, d_out: K of several loads a wave and of less than one, with tails
WEIGHT_SHAPES = [
    (1, 4640, 264), (8, 96, 2056), (1, 544, 4104), (8, 4640, 4104), (3, 96, 8200), (8, 4640, 8200),
    (9, 96, 8184), (12, 544, 2056), (16, 4640, 264),
    (30, 544, 264), (60, 1056, 8136), (256, 544, 4104), (300, 96, 4168), (512, 1056, 2056),
    (1024, 608, 4096), (512, 96, 8192), (1100, 1056, 4104),
    (2100, 512, 8200), (2100, 768, 8200), (2100, 608, 8200),
]
BOTH_SHAPES = [
    (3, 96, 8200), (60, 1056, 8136), (300, 544, 4168), (512, 1056, 2056), (1024, 608, 4096),
    (512, 96, 6144), (256, 1536, 14336), (1024, 1056, 4096), (2100, 512, 8200), (2100, 608, 8200),
]


@pytest.mark.parametrize("n,d_in,d_out", WEIGHT_SHAPES)
def test_weight(n, d_in, d_out):
    say("weight", n, d_in, d_out)
    codes, scales = wl.make_mxfp4(d_out, d_out, d_in)
    X = random_rows(n, d_in + 8, n)[:, :d_in]
    out = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(X, *packed(codes, scales), out[:n, :d_out])
    assert bool((out[n] == 7.0).all()) and bool((out[:, d_out:] == 7.0).all())
    X64, W64 = X.double(), values(codes, scales)
    check(out[:n, :d_out], X64 @ W64.t(), d_in * U * (X64.abs() @ W64.abs().t()), "weight")


@pytest.mark.parametrize("n,d_in,d_out", BOTH_SHAPES)
@pytest.mark.parametrize("pad", [0, 4])
def test_both_operands(n, d_in, d_out, pad):
    say("both", n, d_in, d_out, pad)
    xc, xs = wl.make_mxfp4(n + 1, n, d_in, 124, 130)
    wc, ws = wl.make_mxfp4(d_out, d_out, d_in)
    out = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4(*packed(xc, xs, pad), *packed(wc, ws, pad), out[:n, :d_out])
    assert bool((out[n] == 7.0).all()) and bool((out[:, d_out:] == 7.0).all())
    X64, W64 = values(xc, xs), values(wc, ws)
    check(out[:n, :d_out], X64 @ W64.t(), d_in * U * (X64.abs() @ W64.abs().t()), "both")


# n, d_in, d_out, n_slots, rank bound of a projection
LORA_SHAPES = [
    (8, 544, 2056, 5, 16), (5, 544, 4104, 4, 64), (5, 544, 8200, 4, 32), (12, 544, 2056, 6, 64),
    (30, 96, 2056, 9, 32), (256, 544, 4104, 17, 64), (300, 96, 4168, 5, 16), (1024, 608, 4096, 9, 64),
    (2304, 96, 8192, 7, 32), (2100, 608, 8200, 5, 64), (2048, 608, 8192, 5, 64), (2040, 96, 8136, 7, 16),
]


@pytest.mark.parametrize("n,d_in,d_out,n_slots,r", LORA_SHAPES)
@pytest.mark.parametrize("kind", ["plain", "runs", "no copy of B", "dora", "stacked dora"])
def test_adapters(n, d_in, d_out, n_slots, r, kind):
    """Rows of their own adapter each and requests of many rows, with and without
    the pool's second copy of B, DoRA factors and stacked projections; base-only
    and rank-0 rows bit for bit the base product's."""
    say("adapters", n, d_in, d_out, n_slots, r, kind)
    P = 2 if kind == "stacked dora" else 1
    outs = [d_out // 2 // 8 * 8, d_out - d_out // 2 // 8 * 8] if P > 1 else [d_out]
    dora = "dora" in kind
    ranks = [8, 0] + [min(r, (5, 16, 64, 24)[a % 4]) for a in range(n_slots - 2)]
    parts = [wl.make_random(650 + n + q, n, d_in, o, n_slots, r, ranks=ranks, p_base=0.15, dtype="bf16",
                            runs=kind in ("runs", "stacked dora")) for q, o in enumerate(outs)]
    w = parts[0]
    dev = [wl.device_tensors(p, DEV) for p in parts]
    natural = kind != "no copy of B"
    if P > 1:
        pool = srg.Pool.stacked([srg.Pool(d["A"], d["Bt"], d["slot_rank"], w.slot_alpha) for d in dev],
                                dora=True)
    else:
        pool = srg.Pool(dev[0]["A"], dev[0]["Bt"], dev[0]["slot_rank"], w.slot_alpha, natural_b=natural,
                        dora=dora)
    gen = torch.Generator(DEV).manual_seed(n)
    if dora:
        pool.dora_scale.copy_(0.5 + 1.5 * torch.rand(n_slots, d_out, device=DEV, generator=gen))
    codes, scales = wl.make_mxfp4(651, d_out, d_in)
    Wq, ws = packed(codes, scales)
    X, slot = dev[0]["X"], torch.from_numpy(w.row_slot).to(DEV)
    seg = srg.Segments(n, n_slots, DEV)
    H = torch.full((n, pool.r_max), float("nan"), device=DEV)
    srg.lora_build_shrink(dev[0]["row_slot"], X, pool, seg, H)
    Yf = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_linear_fused_mxfp4w(X, Wq, ws, H, seg, pool, Yf[:n, :d_out])
    assert bool((Yf[n] == 7.0).all()) and bool((Yf[:, d_out:] == 7.0).all())
    Yb = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(X, Wq, ws, Yb)

    X64, W64 = X.double(), values(codes, scales)
    sums = X64.abs() @ W64.abs().t()
    Y64, acc = X64 @ W64.t(), d_in * U * sums
    base = slot < 0
    for a, k in enumerate(ranks):
        rows = (slot == a).nonzero().squeeze(1)
        if k == 0:
            base |= slot == a
            continue
        if not len(rows):
            continue
        s, at = float(w.slot_alpha[a]) / k, 0
        for d, o in zip(dev, outs):
            A, B = d["A"][a, :k].double(), d["Bt"][a, :k].double()
            h, h_abs = X64[rows] @ A.t(), X64[rows].abs() @ A.abs().t()
            c = slice(at, at + o)
            Y64[rows, c] += s * (h @ B)
            acc[rows, c] += s * ((h_abs * (d_in + k + 2) * U + h.abs() * 2.0 ** -16) @ B.abs())
            acc[rows, c] += (2 * k + 2) * U * (sums[rows, c] + s * (h_abs @ B.abs()))
            at += o
        if dora:
            g = pool.dora_scale[a].double()
            Y64[rows] *= g
            acc[rows] = acc[rows] * g + U * Y64[rows].abs()
    check(Yf[:n, :d_out], Y64, acc, kind)
    assert torch.equal(Yf[:n, :d_out][base], Yb[base])


# a shape of each kernel: n, d_out
EACH_WEIGHT = [(1, 264), (3, 4104), (8, 8200), (12, 2056), (30, 264), (300, 4168), (1024, 4096), (2100, 8200)]
EACH_BOTH = [(3, 264), (300, 4168), (1024, 4096), (2100, 8200)]


@pytest.mark.parametrize("n,d_out", EACH_WEIGHT)
@pytest.mark.parametrize("lo,hi,up", [(0, 40, 100), (214, 251, -100)])
def test_weight_scales_over_their_range(n, d_out, lo, hi, up):
    """The least scales, whose values are subnormal in bf16, and the largest with
    all values finite, under activations that bring the products back."""
    say("weight scales", n, d_out, lo, hi)
    d_in = 160
    codes, scales = wl.make_mxfp4(n + lo, d_out, d_in, lo, hi)
    X = random_rows(n, d_in, n) * 2.0 ** up
    out = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(X, *packed(codes, scales), out)
    X64, W64 = X.double(), values(codes, scales)
    check(out, X64 @ W64.t(), d_in * U * (X64.abs() @ W64.abs().t()), "weight scales")


@pytest.mark.parametrize("n,d_out", EACH_BOTH)
@pytest.mark.parametrize("lo,hi", [(0, 40), (214, 254)])
def test_both_scales_over_their_range(n, d_out, lo, hi):
    say("both scales", n, d_out, lo, hi)
    d_in = 160
    xc, xs = wl.make_mxfp4(n + lo, n, d_in, 254 - hi, 254 - lo)
    wc, ws = wl.make_mxfp4(n + hi, d_out, d_in, lo, hi)
    out = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4(*packed(xc, xs), *packed(wc, ws), out)
    X64, W64 = values(xc, xs), values(wc, ws)
    check(out, X64 @ W64.t(), d_in * U * (X64.abs() @ W64.abs().t()), "both scales")


@pytest.mark.parametrize("n,d_out", EACH_WEIGHT)
def test_nan_stays_in_its_row_and_column(n, d_out):
    """NaN scales of W make NaN of their columns, a NaN or an infinity of X of its
    row alone, on every kernel."""
    say("nan", n, d_out)
    d_in = 608
    codes, scales = wl.make_mxfp4(5, d_out, d_in)
    scales[17, 18] = 255
    scales[d_out - 1, 0] = 255
    W = packed(codes, scales)
    X = random_rows(n, d_in, n)
    Y = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    bad = torch.zeros((n, d_out), dtype=torch.bool, device=DEV)
    bad[:, [17, d_out - 1]] = True
    srg.lora_base_gemm_mxfp4w(X, *W, Y)
    assert torch.equal(torch.isnan(Y), bad)
    X[n - 1, 607] = float("nan")
    bad[n - 1] = True
    srg.lora_base_gemm_mxfp4w(X, *W, Y)
    assert torch.equal(torch.isnan(Y), bad)
    X[n - 1, 607] = float("inf")                     # in a quantised row: a NaN block
    Xq = srg.mxfp4_empty(n, d_in)
    srg.lora_mxfp4_quantize(X, *Xq)
    srg.lora_base_gemm_mxfp4(*Xq, *W, Y)
    assert torch.equal(torch.isnan(Y), bad)


# n, top_k, E, d_in, d_out: the persistent kernel's ways of loading scales, and more
# experts than a workgroup has threads
EXPERT_SHAPES = [(4800, 2, 64, 768, 1032), (5000, 2, 64, 512, 1032), (2600, 4, 64, 608, 1032),
                 (12000, 4, 590, 256, 72), (3000, 2, 5, 768, 264), (1500, 4, 9, 608, 136), (30, 4, 8, 2080, 264), (30, 4, 30, 4640, 136), (40, 1, 7, 1056, 520),
                 (150, 4, 100, 544, 776), (500, 4, 1000, 96, 136), (20, 2, 6, 4640, 264)]


@pytest.mark.parametrize("n,k,E,d_in,d_out", EXPERT_SHAPES)
@pytest.mark.parametrize("gathered", [True, False])
def test_experts(n, k, E, d_in, d_out, gathered):
    say("experts", n, k, E, d_in, d_out, gathered)
    ids = np.random.default_rng(n + E).integers(-1, E, size=(n, k)).astype(np.int32)
    ref = oracle.expert_routing(ids, E)
    order, off = ref["sorted_choice"], ref["expert_offsets"]
    ex = srg.Experts(n, k, E, DEV)
    srg.lora_experts_sort(torch.from_numpy(ids).to(DEV), ex)
    codes, scales = wl.make_mxfp4(E + d_out, E * d_out, d_in)
    Wq, ws = packed(codes, scales)
    ws = ws.as_strided((E, d_out, d_in // 32), (d_out * ws.stride(0), ws.stride(0), 1))
    X = random_rows(n if gathered else n * k, d_in, n)
    Y = torch.full((n * k, d_out), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_experts_gemm_mxfp4w(X, ex, Wq.view(E, d_out, d_in // 2), ws, Y, gathered=gathered)
    assert bool((Y[len(order):] == 7.0).all())
    rows = torch.from_numpy(order // k if gathered else np.arange(len(order))).long().to(DEV)
    Y64, acc = (torch.zeros((len(order), d_out), dtype=torch.float64, device=DEV) for _ in range(2))
    for e in range(E):
        p = slice(int(off[e]), int(off[e + 1]))
        W64 = values(codes[e * d_out:(e + 1) * d_out], scales[e * d_out:(e + 1) * d_out])
        X64 = X[rows[p]].double()
        Y64[p] = X64 @ W64.t()
        acc[p] = d_in * U * (X64.abs() @ W64.abs().t())
    check(Y[:len(order)], Y64, acc, "experts")


def test_segments_on_the_host_are_refused():
    n, d_in, d_out = 5, 64, 16
    w = wl.make_random(3, n, d_in, d_out, 2, 8, dtype="bf16")
    d = wl.device_tensors(w, DEV)
    pool = srg.Pool(d["A"], d["Bt"], d["slot_rank"], w.slot_alpha)
    Wq, ws = srg.mxfp4_empty(d_out, d_in, DEV)
    Y = torch.full((n, d_out), 7.0, dtype=torch.bfloat16, device=DEV)
    H = torch.zeros((n, 8), device=DEV)
    with pytest.raises(ValueError):
        srg.lora_linear_fused_mxfp4w(d["X"], Wq, ws, H, srg.Segments(n, 2, "cpu"), pool, Y)
    assert bool((Y == 7.0).all())


@pytest.mark.parametrize("n,d_in,d_out,n_slots,r,runs", [
    (9, 544, 264, 4, 16, False), (300, 544, 4168, 7, 64, True), (300, 1056, 4168, 40, 32, False),
    (1024, 608, 4096, 9, 64, True), (2100, 512, 8200, 5, 64, True)])
def test_two_mxfp4_operands_with_adapters(n, d_in, d_out, n_slots, r, runs):
    """quantise, build and shrink, the product of the codes, expand: the term comes
    from the unquantised activations and is added to the rounded product, so two
    roundings to bf16, of the base and of the sum."""
    say("both with adapters", n, d_in, d_out, n_slots, r, runs)
    w = wl.make_random(660 + n, n, d_in, d_out, n_slots, r, p_base=0.15, dtype="bf16", runs=runs)
    w.slot_rank[1] = 0
    d = wl.device_tensors(w, DEV)
    pool = srg.Pool(d["A"], d["Bt"], d["slot_rank"], w.slot_alpha)
    seg = srg.Segments(n, n_slots, DEV)
    H = torch.full((n, r), float("nan"), device=DEV)
    X, slot = d["X"], torch.from_numpy(w.row_slot).to(DEV)
    codes, scales = wl.make_mxfp4(661, d_out, d_in)
    W = packed(codes, scales)
    Xq = srg.mxfp4_empty(n, d_in)
    Y = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_mxfp4_quantize(X, *Xq)
    srg.lora_build_shrink(d["row_slot"], X, pool, seg, H)
    srg.lora_base_gemm_mxfp4(*Xq, *W, Y[:n, :d_out])
    base = Y.clone()
    srg.lora_expand(H, seg, pool, Y[:n, :d_out])
    assert bool((Y[n] == 7.0).all()) and bool((Y[:, d_out:] == 7.0).all())

    Xd = values(*oracle.quantize_mxfp4(X.double().cpu().numpy()))
    W64, X64 = values(codes, scales), X.double()
    sums = Xd.abs() @ W64.abs().t()
    Y64, acc = Xd @ W64.t(), d_in * U * sums
    check(base[:n, :d_out], Y64, acc, "base")
    acc += 2.0 ** -8 * Y64.abs()                         # the base's own rounding
    plain = slot < 0
    for a in range(n_slots):
        k, rows = int(w.slot_rank[a]), (slot == a).nonzero().squeeze(1)
        if k == 0:
            plain |= slot == a
            continue
        s = float(w.slot_alpha[a]) / k
        A, B = d["A"][a, :k].double(), d["Bt"][a, :k].double()
        h, h_abs = X64[rows] @ A.t(), X64[rows].abs() @ A.abs().t()
        Y64[rows] += s * (h @ B)
        acc[rows] += s * ((h_abs * (d_in + k + 2) * U + h.abs() * 2.0 ** -16) @ B.abs())
        acc[rows] += (2 * k + 2) * U * (sums[rows] + s * (h_abs @ B.abs()))
    check(Y[:n, :d_out], Y64, acc, "sum")
    assert torch.equal(Y[:n][plain], base[:n][plain])


def test_experts_layer_in_a_graph_against_float64():
    """An expert layer (sort, two products, combine, the combine's gradients),
    captured once and replayed on new inputs: each call's output against float64
    from the stored inputs of that call."""
    n, k, E, d, f = 72, 4, 9, 160, 96
    c1, s1 = wl.make_mxfp4(31, E * 2 * f, d, 120, 124)
    c2, s2 = wl.make_mxfp4(32, E * d, f, 120, 124)
    W1, W2 = values(c1, s1).view(E, 2 * f, d), values(c2, s2).view(E, d, f)
    (q1, w1), (q2, w2) = packed(c1, s1), packed(c2, s2)
    q1, q2 = q1.view(E, 2 * f, d // 2), q2.view(E, d, f // 2)
    w1 = w1.as_strided((E, 2 * f, d // 32), (2 * f * w1.stride(0), w1.stride(0), 1))
    w2 = w2.as_strided((E, d, f // 32), (d * w2.stride(0), w2.stride(0), 1))
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)   # noqa: E731
    X, dY, h, a, y, out, dys = z(n, d), z(n, d), z(n * k, 2 * f), z(n * k, f), z(n * k, d), z(n, d), z(n * k, d)
    ids, wt, dw = z(n, k, t=torch.int32), z(n, k, t=torch.float32), z(n, k, t=torch.float32)
    ex = srg.Experts(n, k, E, DEV)

    def step():
        srg.lora_experts_sort(ids, ex)
        srg.lora_experts_gemm_mxfp4w(X, ex, q1, w1, h)
        a.copy_(torch.nn.functional.silu(h[:, :f].float()) * h[:, f:].float())
        srg.lora_experts_gemm_mxfp4w(a, ex, q2, w2, y, gathered=False)
        srg.lora_experts_combine(y, wt, ex, out)
        srg.lora_experts_combine_backward(dY, y, wt, ex, dys, dw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        say("graph", rep)
        host = np.random.default_rng(rep).integers(-1, E, size=(n, k)).astype(np.int32)
        ids.copy_(torch.from_numpy(host))
        g = torch.Generator(DEV).manual_seed(rep)
        for t in (X, dY, wt):
            t.copy_(torch.randn(t.shape, device=DEV, generator=g))
        for t in (h, y, dys):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle.expert_routing(host, E)
        order, off = ref["sorted_choice"], ref["expert_offsets"]
        kept = len(order)
        assert np.array_equal(ex.choice_position.cpu().numpy(), ref["choice_position"])
        tok = torch.from_numpy(order // k).long().to(DEV)
        expert = torch.from_numpy(np.repeat(np.arange(E), np.diff(off))).to(DEV)
        x64, a64, y64 = X[tok].double(), a[:kept].double(), y[:kept].double()

        def product(v, W):
            r = [torch.zeros((kept, W.shape[1]), dtype=torch.float64, device=DEV) for _ in range(2)]
            for e in range(E):
                m = expert == e
                r[0][m], r[1][m] = v[m] @ W[e].t(), v.shape[1] * U * (v[m].abs() @ W[e].abs().t())
            return r
        check(h[:kept], *product(x64, W1), "h")
        check(y[:kept], *product(a64, W2), "y")
        wc = wt.double().reshape(-1)[torch.from_numpy(order).long().to(DEV)]
        o64, o_abs = (torch.zeros((n, d), dtype=torch.float64, device=DEV).index_add_(0, tok, t)
                      for t in (wc[:, None] * y64, (wc[:, None] * y64).abs()))
        check(out, o64, (k + 1) * U * o_abs, "out")
        dy64 = dY[tok].double()
        check(dys[:kept], wc[:, None] * dy64, U * (wc[:, None] * dy64).abs(), "dys")
        flat = torch.zeros(n * k, dtype=torch.float64, device=DEV)
        bound = flat.clone()
        at = torch.from_numpy(order).long().to(DEV)
        flat[at], bound[at] = (dy64 * y64).sum(1), (d + 2) * U * (dy64 * y64).abs().sum(1)
        assert bool(((dw.double().reshape(-1) - flat).abs() <= bound).all())
        for t in (h, y, dys):
            assert bool((t[kept:] == 3.0).all())
