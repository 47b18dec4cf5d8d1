"""GPU parity of MXFP4: quantising and back bit for bit against the oracle, and
the products with MXFP4 operands (an MXFP4 weight with and without the LoRA
term, both operands MXFP4) elementwise against float64.

Tolerance of a product's element: its own rounding to bf16, 2^-8 |y|, plus the
fp32 accumulation.  A sum of K products in fp32, in any order and grouping,
each addition off by at most one unit of 2^-23 relative to the partial sum
(rounded or cut off), is off by at most K 2^-23 sum |x_c w_c|; the products
themselves are exact in fp32 (8 + 3 bits).  The LoRA term adds its H's sum over
d_in, its own sum over r, the scale's product, and the split of s H into two
bf16 parts (2^-16 relative)."""
import numpy as np
import pytest
import torch

import oracle
import segmented_rank_gemm_segment_amd as srg
import workloads as wl
from gpu_harness import DEV, say, to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    srg.lib()
    yield
    torch.cuda.synchronize()


def mx_device(codes, scales, pad_byte=255):
    """Codes and scales on the device, both with padded rows whose padding
    (NaN scales) must never be used."""
    n, hb = codes.shape
    g = scales.shape[1]
    c = torch.full((n, hb + 16), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((n, (g + 3) // 4 * 4 + 4), pad_byte, dtype=torch.uint8, device=DEV)
    c[:, :hb] = torch.from_numpy(codes).to(DEV)
    s[:, :g] = torch.from_numpy(scales).to(DEV)
    return c[:, :hb], s[:, :g]


def bf16_device(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).to(DEV).view(torch.bfloat16)


def check_close(Y, Y64, tol, what):
    d = np.abs(to_f64(Y) - Y64)
    worst = float(np.max(d / np.maximum(tol, 1e-300))) if d.size else 0.0
    say(what, "worst error / tolerance", worst)
    assert np.all(d <= tol), (what, worst)


def product_tol(X64, W64, Y64):
    return 2.0 ** -8 * np.abs(Y64) + X64.shape[1] * U * (np.abs(X64) @ np.abs(W64).T)


# ---------------------------------------------------------------------------
# quantise and back
# ---------------------------------------------------------------------------
def rows_of_all_kinds(seed, n, d, dtype):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)).astype(np.float32) * \
        np.exp2(rng.integers(-8, 8, size=(n, 1))).astype(np.float32)
    blk = x.reshape(n * d // 32, 32)
    kinds = rng.integers(0, 9, size=len(blk))
    blk[kinds == 1] = 0
    blk[kinds == 2] = np.round(blk[kinds == 2] * 8) / 8            # ties
    blk[kinds == 3] *= np.float32(2.0 ** -120)                     # near the least scale
    blk[kinds == 4] *= np.float32(2.0 ** -140)                     # subnormal
    with np.errstate(over="ignore"):
        blk[kinds == 5] *= np.float32(2.0 ** 118)                  # near the largest
    for b in np.flatnonzero(kinds == 6)[:3]:
        blk[b, 5] = [np.nan, np.inf, -np.inf][b % 3]
    blk[kinds == 7] = -blk[kinds == 7] * 0
    t = torch.from_numpy(x).to(DEV).to(dtype)
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 32), (3, 64), (257, 96), (5, 2080), (37, 4096)])
def test_quantize_and_back_are_exact(n, d, dtype):
    x, x64 = rows_of_all_kinds(n + d, n, d, dtype)
    wide = torch.full((n, d + 8), 3.0, dtype=dtype, device=DEV)
    wide[:, :d] = x
    qw = torch.full((n, d // 2 + 16), 0xAB, dtype=torch.uint8, device=DEV)
    sw = torch.full((n, (d // 32 + 3) // 4 * 4 + 4), 0xCD, dtype=torch.uint8, device=DEV)
    srg.lora_mxfp4_quantize(wide[:, :d], qw[:, :d // 2], sw[:, :d // 32])
    q, s = oracle.quantize_mxfp4(x64)
    assert np.array_equal(sw[:, :d // 32].cpu().numpy(), s)
    assert np.array_equal(qw[:, :d // 2].cpu().numpy(), q)
    assert bool((qw[:, d // 2:] == 0xAB).all()) and bool((sw[:, d // 32:] == 0xCD).all())
    out = torch.full((n, d + 8), 9.0, dtype=dtype, device=DEV)
    srg.lora_mxfp4_dequantize(qw[:, :d // 2], sw[:, :d // 32], out[:, :d])
    v = oracle.decode_mxfp4(q, s)
    assert np.array_equal(out[:, :d].double().cpu().numpy(), v, equal_nan=True)
    assert bool((out[:, d:] == 9.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_every_code_and_scale(dtype):
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    out = torch.empty((256, 32), dtype=dtype, device=DEV)
    srg.lora_mxfp4_dequantize(torch.from_numpy(codes).to(DEV), mx_device(codes, scales)[1], out)
    with np.errstate(over="ignore"):
        want = oracle.decode_mxfp4(codes, scales)
        # rows of values past the type's range: the type's largest is below 2^128
        want[np.abs(want) >= 2.0 ** 128] *= np.inf
    assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)


def test_no_rows_is_a_no_op():
    q, s = srg.mxfp4_empty(0, 64, DEV)
    x = torch.empty((0, 64), device=DEV)
    srg.lora_mxfp4_quantize(x, q, s)
    srg.lora_mxfp4_dequantize(q, s, x)
    Wq, ws = srg.mxfp4_empty(8, 64, DEV)
    Y = torch.empty((0, 8), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(x.bfloat16(), Wq, ws, Y)
    srg.lora_base_gemm_mxfp4(q, s, Wq, ws, Y)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
SHAPES = [
    # n, d_in, d_out: one row; below one tile; K tails of every kind (d_in mod
    # 512 in blocks of 32); ragged n and d_out; each tile size
    (1, 32, 8), (1, 4096, 264), (2, 96, 16), (5, 1056, 40), (16, 512, 64), (17, 544, 72),
    (33, 2080, 200), (64, 1024, 128), (100, 160, 264), (300, 736, 264), (512, 256, 384),
    (700, 224, 136), (1100, 352, 520), (1100, 96, 8200), (2040, 288, 7944),
    # 32-row tiles: up to 32 rows, and few tiles of 64
    (12, 544, 8200), (16, 96, 16392), (25, 1056, 8200), (32, 2080, 200), (60, 800, 8136),
]


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_weight_product(n, d_in, d_out):
    w = wl.make_random(n + d_in, n, d_in, 8, 1, 8, dtype="bf16")
    codes, scales = wl.make_mxfp4(d_out, d_out, d_in)
    Wq, ws = mx_device(codes, scales)
    ldx = torch.full((n, d_in + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    ldx[:, :d_in] = bf16_device(w.X)
    out = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(ldx[:, :d_in], Wq, ws, out[:n, :d_out])
    X64, W64 = oracle.decode(w.X, "bf16"), oracle.decode_mxfp4(codes, scales)
    Y64 = X64 @ W64.T
    check_close(out[:n, :d_out], Y64, product_tol(X64, W64, Y64), f"weight {n, d_in, d_out}")
    assert bool((out[n] == 7.0).all()) and bool((out[:, d_out:] == 7.0).all())


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_both_operands_product(n, d_in, d_out):
    xc, xs = wl.make_mxfp4(n + 1, n, d_in, 124, 130)
    wc, wsc = wl.make_mxfp4(d_out, d_out, d_in)
    Xq, xsd = mx_device(xc, xs)
    Wq, wsd = mx_device(wc, wsc)
    out = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4(Xq, xsd, Wq, wsd, out[:n, :d_out])
    X64, W64 = oracle.decode_mxfp4(xc, xs), oracle.decode_mxfp4(wc, wsc)
    Y64 = X64 @ W64.T
    check_close(out[:n, :d_out], Y64, product_tol(X64, W64, Y64), f"both {n, d_in, d_out}")
    assert bool((out[n] == 7.0).all()) and bool((out[:, d_out:] == 7.0).all())


@pytest.mark.parametrize("n,d_in,d_out", [
    (2100, 512, 8200), (2100, 1536, 8200), (2100, 96, 8200), (2100, 640, 8200), (4200, 1024, 4104),
    (8200, 512, 256), (700, 2560, 136), (60, 1024, 72)])
@pytest.mark.parametrize("pad", [0, 12])
def test_both_operands_many_tiles(n, d_in, d_out, pad):
    """More output tiles than compute units, scale rows with and without 16-byte
    alignment, and K of one to many stages; every element."""
    xc, xs = wl.make_mxfp4(n + 1, n, d_in, 124, 130)
    wc, wsc = wl.make_mxfp4(d_out, d_out, d_in)
    dev = []
    for c, s in ((xc, xs), (wc, wsc)):
        q = torch.from_numpy(c).to(DEV)
        sp = torch.full((len(s), (s.shape[1] + 15) // 16 * 16 + pad), 255, dtype=torch.uint8, device=DEV)
        sp[:, :s.shape[1]] = torch.from_numpy(s).to(DEV)
        dev += [q, sp[:, :s.shape[1]]]
    out = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4(*dev, out[:n, :d_out])
    assert bool((out[n] == 7.0).all()) and bool((out[:, d_out:] == 7.0).all())
    X64 = torch.from_numpy(oracle.decode_mxfp4(xc, xs)).to(DEV)
    W64 = torch.from_numpy(oracle.decode_mxfp4(wc, wsc)).to(DEV)
    Y64 = X64 @ W64.t()
    tol = 2.0 ** -8 * Y64.abs() + d_in * U * (X64.abs() @ W64.abs().t())
    assert bool(((out[:n, :d_out].double() - Y64).abs() <= tol).all())


def packed(codes, scales, pad=0):
    """On the device, scale rows a multiple of 16 bytes apart plus pad; what
    pads them (NaN scales) must never be used."""
    q = torch.from_numpy(codes).to(DEV)
    s = torch.full((len(scales), (scales.shape[1] + 15) // 16 * 16 + pad), 255, dtype=torch.uint8,
                   device=DEV)
    s[:, :scales.shape[1]] = torch.from_numpy(scales).to(DEV)
    return q, s[:, :scales.shape[1]]


@pytest.mark.parametrize("n,d_in,d_out", [
    (2100, 512, 8200), (2100, 1536, 8200), (2100, 32, 8200), (2100, 64, 8200), (2100, 96, 8200),
    (2100, 128, 8200), (2100, 608, 8200), (2100, 704, 8200), (4200, 1024, 4104), (8200, 640, 2056)])
@pytest.mark.parametrize("pad", [0, 12])
def test_weight_many_tiles(n, d_in, d_out, pad):
    """More output tiles than compute units, scale rows with and without 16-byte
    alignment, K of one stage to many with every tail; every element."""
    codes, scales = wl.make_mxfp4(d_out, d_out, d_in)
    X = torch.randn(n, d_in, device=DEV, generator=torch.Generator(DEV).manual_seed(n)).bfloat16()
    out = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(X, *packed(codes, scales, pad), out[:n, :d_out])
    assert bool((out[n] == 7.0).all()) and bool((out[:, d_out:] == 7.0).all())
    X64, W64 = X.double(), torch.from_numpy(oracle.decode_mxfp4(codes, scales)).to(DEV)
    Y64 = X64 @ W64.t()
    tol = 2.0 ** -8 * Y64.abs() + d_in * U * (X64.abs() @ W64.abs().t())
    assert bool(((out[:n, :d_out].double() - Y64).abs() <= tol).all())


LORA_CASES = [
    # seed, n, d_in, d_out, n_slots, r_max, p_base, runs
    (601, 1, 64, 72, 3, 8, 0.0, False),
    (602, 7, 160, 200, 5, 16, 0.3, False),
    (603, 40, 1056, 136, 40, 64, 0.1, False),
    (604, 300, 544, 264, 40, 64, 0.1, False),
    (605, 512, 256, 384, 6, 32, 0.2, True),
    (606, 700, 224, 136, 7, 64, 0.1, True),
    (607, 1100, 96, 8200, 7, 64, 0.1, True),
    (608, 2040, 96, 7944, 7, 32, 0.1, True),
    (609, 20, 544, 264, 9, 64, 0.2, False),
    (610, 12, 96, 8200, 5, 32, 0.2, False),
    (611, 60, 608, 8136, 20, 16, 0.1, False),
]


def lora_tol(w, X64, W64, Y64, rows):
    """Elementwise tolerance of the fused output (module docstring)."""
    tol = product_tol(X64, W64, Y64)
    for t, i in enumerate(rows):
        a = int(w.row_slot[i])
        r = int(w.slot_rank[a]) if a >= 0 else 0
        if r == 0:
            continue
        A = oracle.decode(w.A[a, :r], "bf16")
        B = np.abs(oracle.decode(w.B[a][:, :r], "bf16"))
        s = float(w.slot_alpha[a]) / r
        h_abs = np.abs(A) @ np.abs(X64[t])
        h = np.abs(A @ X64[t])
        tol[t] += s * (B @ (h_abs * (X64.shape[1] + r + 2) * U + h * 2.0 ** -16))
        # the base sum and the term meet in one fp32 addition per rank step
        tol[t] += (2 * r + 2) * U * (np.abs(W64) @ np.abs(X64[t]) + s * (B @ h_abs))
    return tol


@pytest.mark.parametrize("case", LORA_CASES, ids=[f"s{c[0]}" for c in LORA_CASES])
@pytest.mark.parametrize("natural_b", [True, False])
def test_fused_lora(case, natural_b):
    seed, n, d_in, d_out, n_slots, r_max, p_base, runs = case
    w = wl.make_random(seed, n, d_in, d_out, n_slots, r_max, p_base=p_base, dtype="bf16", runs=runs)
    if n_slots > 2:
        w.slot_rank[1] = 0
    codes, scales = wl.make_mxfp4(seed, d_out, d_in)
    Wq, ws = mx_device(codes, scales)
    d = wl.device_tensors(w, DEV)
    pool = srg.Pool(d["A"], d["Bt"], d["slot_rank"], w.slot_alpha, natural_b=natural_b)
    seg = srg.Segments(w.n, w.n_slots, DEV)
    H = torch.full((n, r_max), float("nan"), device=DEV)
    srg.lora_build_shrink(d["row_slot"], d["X"], pool, seg, H)
    Yf = torch.full((n, d_out), float("nan"), dtype=torch.bfloat16, device=DEV)
    srg.lora_linear_fused_mxfp4w(d["X"], Wq, ws, H, seg, pool, Yf)
    Yb = torch.empty_like(Yf)
    srg.lora_base_gemm_mxfp4w(d["X"], Wq, ws, Yb)
    rows = sorted(set(np.random.default_rng(seed).integers(0, n, 128).tolist()) | {0, n - 1})
    Y64, dY64, _ = oracle.lora_forward_mxfp4w(w.X, codes, scales, w.A, w.B, w.row_slot, w.slot_rank,
                                              w.slot_alpha, r_max, "bf16", rows=rows)
    X64, W64 = oracle.decode(w.X, "bf16")[rows], oracle.decode_mxfp4(codes, scales)
    ti = torch.as_tensor(rows, device=DEV)
    check_close(Yf[ti], Y64, lora_tol(w, X64, W64, Y64, rows), f"lora {case}")
    base = torch.as_tensor([i for i in range(n) if w.row_slot[i] < 0
                            or int(w.slot_rank[w.row_slot[i]]) == 0], device=DEV, dtype=torch.long)
    assert torch.equal(Yf[base], Yb[base])
    assert bool(torch.isfinite(Yf.float()).all())


@pytest.mark.parametrize("n", [3, 40, 600])
def test_dora_and_stacked_pools(n):
    """DoRA factors and stacked projections reach the MXFP4 product as they do
    the bf16 one: equal weights in both formats give two fp32 sums of the same
    terms, each within its accumulation bound and one bf16 rounding."""
    d_in, outs, r = 128, [64, 72], 16
    ranks = [16, 8, 16, 16]
    ws_, pools = [], []
    for q, d_out in enumerate(outs):
        w = wl.make_random(620 + q, n, d_in, d_out, 4, r, ranks=ranks, dtype="bf16", pad="zero")
        d = wl.device_tensors(w, DEV)
        pools.append(srg.Pool(d["A"], d["Bt"], d["slot_rank"], w.slot_alpha))
        ws_.append(w)
        if q == 0:
            first = d
    pool = srg.Pool.stacked(pools, dora=True)
    pool.dora_scale[1].fill_(2.0)                        # an exact factor
    codes, scales = wl.make_mxfp4(621, sum(outs), d_in)
    Wq, ws = mx_device(codes, scales)
    W = torch.from_numpy(oracle.decode_mxfp4(codes, scales)).to(DEV).bfloat16()
    seg = srg.Segments(n, 4, DEV)
    H = torch.zeros((n, pool.r_max), device=DEV)
    srg.lora_build_shrink(first["row_slot"], first["X"], pool, seg, H)
    Y1 = torch.empty((n, sum(outs)), dtype=torch.bfloat16, device=DEV)
    Y2 = torch.empty_like(Y1)
    srg.lora_linear_fused(first["X"], W, H, seg, pool, Y1)
    srg.lora_linear_fused_mxfp4w(first["X"], Wq, ws, H, seg, pool, Y2)
    X64, W64 = np.abs(to_f64(first["X"])), np.abs(oracle.decode_mxfp4(codes, scales))
    sums = X64 @ W64.T                                   # sum of the terms' magnitudes
    term = np.zeros_like(sums)
    for i in range(n):
        a = int(ws_[0].row_slot[i])
        if a >= 0:
            k = ranks[a]
            term[i] = 16.0 / k * np.concatenate(
                [np.abs(oracle.decode(w.B[a][:, :k], "bf16")) @ (np.abs(oracle.decode(w.A[a, :k], "bf16")) @ X64[i])
                 for w in ws_])
    one = 2.0 ** -8 * np.abs(to_f64(Y1)) + 2 * ((d_in + 3 * r + 8) * U * (sums + term) + 2.0 ** -16 * term)
    check_close(Y2, to_f64(Y1), 2.02 * one, f"dora, stacked {n}")


@pytest.mark.parametrize("n", [1, 40, 600])
def test_exact_on_small_integers(n):
    """Integer operands whose sums stay below 2^8: every product and sum is
    exact and so is the bf16 result."""
    rng = np.random.default_rng(n)
    d_in, d_out = 64, 136
    x = rng.integers(-1, 2, size=(n, d_in))
    X = torch.from_numpy(x.astype(np.float32)).to(DEV).bfloat16()
    wv = rng.integers(-2, 3, size=(d_out, d_in))
    code = np.array([0, 2, 4])[np.abs(wv)] | np.where(wv < 0, 8, 0)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    scales = np.full((d_out, 2), 127, np.uint8)
    Wq, ws = mx_device(codes, scales)
    Y = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(X, Wq, ws, Y)
    assert np.array_equal(to_f64(Y), (x @ wv.T).astype(np.float64))
    Xq, xs = srg.mxfp4_empty(n, d_in, DEV)
    srg.lora_mxfp4_quantize(X, Xq, xs)
    srg.lora_base_gemm_mxfp4(Xq, xs, Wq, ws, Y)
    assert np.array_equal(to_f64(Y), (x @ wv.T).astype(np.float64))


@pytest.mark.parametrize("n", [1, 20, 300, 1100])
def test_nan_scales_stay_in_their_row(n):
    d_in, d_out = 160, 200
    w = wl.make_random(n, n, d_in, 8, 1, 8, dtype="bf16")
    codes, scales = wl.make_mxfp4(5, d_out, d_in)
    scales[17, 4] = 255
    scales[199, 0] = 255
    Wq, ws = mx_device(codes, scales)
    X = bf16_device(w.X)
    Y = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(X, Wq, ws, Y)
    nan = torch.isnan(Y)
    assert bool(nan[:, [17, 199]].all()) and int(nan.sum()) == 2 * n
    Xq, xs = srg.mxfp4_empty(n, d_in, DEV)
    X[n - 1, 3] = float("inf")
    srg.lora_mxfp4_quantize(X, Xq, xs)
    srg.lora_base_gemm_mxfp4(Xq, xs, Wq, ws, Y)
    nan = torch.isnan(Y)
    assert bool(nan[:, [17, 199]].all()) and bool(nan[n - 1].all())
    assert int(nan.sum()) == 2 * n + d_out - 2


def test_quantize_then_product_on_another_stream_and_in_a_graph():
    """The calls in the order a layer makes them, captured once and replayed on
    new inputs, each replay against eager calls on another stream."""
    n, d_in, d_out = 96, 512, 264
    wc, wsc = wl.make_mxfp4(9, d_out, d_in)
    Wq, ws = mx_device(wc, wsc)
    X = torch.zeros((n, d_in), dtype=torch.bfloat16, device=DEV)
    Xq, xs = srg.mxfp4_empty(n, d_in, DEV)
    Y, Yw = (torch.zeros((n, d_out), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step(x, q, s, y, yw):
        srg.lora_mxfp4_quantize(x, q, s)
        srg.lora_base_gemm_mxfp4(q, s, Wq, ws, y)
        srg.lora_base_gemm_mxfp4w(x, Wq, ws, yw)

    step(X, Xq, xs, Y, Yw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(X, Xq, xs, Y, Yw)
    side = torch.cuda.Stream()
    for k in range(4):
        X.copy_(torch.randn(n, d_in, device=DEV, generator=torch.Generator(DEV).manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q2, s2 = srg.mxfp4_empty(n, d_in, DEV)
            y2, yw2 = torch.empty_like(Y), torch.empty_like(Yw)
            step(X, q2, s2, y2, yw2)
        side.synchronize()
        assert torch.equal(Y, y2) and torch.equal(Yw, yw2) and torch.equal(Xq, q2)
        assert float(Y.abs().max()) > 0


@pytest.mark.parametrize("n,d_in,d_out,n_slots,r_max", [
    (2100, 512, 8200, 7, 64), (2100, 96, 8200, 16, 16), (2100, 640, 8200, 5, 8), (2304, 128, 8192, 17, 32),
    (2040, 1024, 8200, 3, 32), (3100, 96, 5120, 9, 64)])
@pytest.mark.parametrize("runs", [True, False])
def test_fused_lora_many_tiles(n, d_in, d_out, n_slots, r_max, runs):
    """The large batches' LoRA term, requests of many rows and rows of their own
    adapter each, more tiles than compute units; every element, and the
    base-only rows bit for bit the base product's."""
    w = wl.make_random(640 + n_slots, n, d_in, d_out, n_slots, r_max, p_base=0.1, dtype="bf16", runs=runs)
    w.slot_rank[1] = 0
    if r_max > 8:
        w.slot_rank[2] = 5                               # a rank that is no multiple of 8
    codes, scales = wl.make_mxfp4(641, d_out, d_in)
    Wq, ws = packed(codes, scales)
    d = wl.device_tensors(w, DEV)
    pool = srg.Pool(d["A"], d["Bt"], d["slot_rank"], w.slot_alpha)
    seg = srg.Segments(w.n, w.n_slots, DEV)
    H = torch.full((n, r_max), float("nan"), device=DEV)
    srg.lora_build_shrink(d["row_slot"], d["X"], pool, seg, H)
    Yf = torch.full((n + 1, d_out + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_linear_fused_mxfp4w(d["X"], Wq, ws, H, seg, pool, Yf[:n, :d_out])
    assert bool((Yf[n] == 7.0).all()) and bool((Yf[:, d_out:] == 7.0).all())
    Yb = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    srg.lora_base_gemm_mxfp4w(d["X"], Wq, ws, Yb)
    X64, W64 = d["X"].double(), torch.from_numpy(oracle.decode_mxfp4(codes, scales)).to(DEV)
    sums = X64.abs() @ W64.abs().t()
    Y64 = X64 @ W64.t()
    tol = torch.zeros_like(Y64)
    slot = torch.from_numpy(w.row_slot).to(DEV)
    base = slot < 0
    for a in range(n_slots):
        r, rows = int(w.slot_rank[a]), (slot == a).nonzero().squeeze(1)
        if r == 0:
            base |= slot == a
            continue
        s = float(w.slot_alpha[a]) / r
        A, B = d["A"][a, :r].double(), d["Bt"][a, :r].double()
        h, h_abs = X64[rows] @ A.t(), X64[rows].abs() @ A.abs().t()
        Y64[rows] += s * (h @ B)
        # H's sum, its split and the term's own sum, as in lora_tol
        tol[rows] += s * ((h_abs * (d_in + r + 2) * U + h.abs() * 2.0 ** -16) @ B.abs())
        tol[rows] += (2 * r + 2) * U * (sums[rows] + s * (h_abs @ B.abs()))
    tol += 2.0 ** -8 * Y64.abs() + d_in * U * sums
    assert bool(((Yf[:n, :d_out].double() - Y64).abs() <= tol).all())
    assert torch.equal(Yf[:n, :d_out][base], Yb[base])


@pytest.mark.parametrize("n,d_in,d_out", [
    (40, 256, 4104), (130, 512, 4096), (300, 1024, 4168), (500, 1536, 2056),
    (2100, 64, 8200), (2100, 128, 8192), (2100, 192, 8200), (2300, 512, 8200)])
@pytest.mark.parametrize("x_is_mx", [False, True])
def test_short_k_fresh_operands_repeated(n, d_in, d_out, x_is_mx):
    """One to a few stages of K on operands copied right before the call, three
    times: a stage is read only after all of its loads have landed, cold ones
    too, whatever order they land in."""
    xc, xs = wl.make_mxfp4(n + 1, n, d_in, 124, 130)
    wc, wsc = wl.make_mxfp4(d_out, d_out, d_in)
    X64 = torch.from_numpy(oracle.decode_mxfp4(xc, xs)).to(DEV)
    W64 = torch.from_numpy(oracle.decode_mxfp4(wc, wsc)).to(DEV)
    Y64 = X64 @ W64.t()
    tol = 2.0 ** -8 * Y64.abs() + d_in * U * (X64.abs() @ W64.abs().t())
    Xb = X64.bfloat16().cpu()                       # exact: codes of 2 significant bits
    for rep in range(3):
        say("fresh", n, d_in, d_out, x_is_mx, rep)
        W = packed(wc, wsc)
        out = torch.full((n, d_out), 7.0, dtype=torch.bfloat16, device=DEV)
        if x_is_mx:
            srg.lora_base_gemm_mxfp4(*packed(xc, xs), *W, out)
        else:
            srg.lora_base_gemm_mxfp4w(Xb.to(DEV), *W, out)
        assert bool(((out.double() - Y64).abs() <= tol).all()), rep


def test_two_streams_at_once():
    """Products of every size on two streams at the same time, each with its
    own operands and outputs: the bits of one call after the other."""
    d_in, d_out = 544, 2056
    calls = []
    for n in (3, 12, 30, 200, 700, 2100):
        wc, wsc = wl.make_mxfp4(n, d_out, d_in)
        W = packed(wc, wsc)
        X = torch.randn(n, d_in, device=DEV, generator=torch.Generator(DEV).manual_seed(n)).bfloat16()
        Xq = srg.mxfp4_empty(n, d_in)
        srg.lora_mxfp4_quantize(X, *Xq)
        calls.append((X, Xq, W))
    def outputs():
        return [[torch.full((len(X), d_out), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
                for X, _, _ in calls]
    def run(outs, order, stream):
        for i in order:
            X, Xq, W = calls[i]
            srg.lora_base_gemm_mxfp4w(X, *W, outs[i][0], stream=stream)
            srg.lora_base_gemm_mxfp4(*Xq, *W, outs[i][1], stream=stream)
    want = outputs()
    run(want, range(len(calls)), None)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        a, b = outputs(), outputs()
        torch.cuda.synchronize()
        run(a, range(len(calls)), s1)
        run(b, reversed(range(len(calls))), s2)
        torch.cuda.synchronize()
        for got in (a, b):
            for g, w in zip(got, want):
                assert all(torch.equal(x, y) for x, y in zip(g, w)), rep
