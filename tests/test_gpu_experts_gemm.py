"""The experts' products on bf16 weights and their gradients against float64.

Tolerance: bf16 products are exact in fp32, and a sum of k of them is off by at
most (k + 8) 2^-24 times the sum of their magnitudes in any order; the result is
rounded once, by at most 2^-8 (bf16) or 2^-24 (fp32) of it, after an old value is
added in fp32 (one rounding more)."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg
from gpu_harness import DEV, say
from test_gpu_experts import make_ids, sorted_batch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


def rows_of(rows, width, pad, fill=float("nan")):
    return torch.full((rows, width + pad), fill, dtype=BF, device=DEV)[:, :width]


def matrices(E, d_out, d_in, pad, dtype=BF, fill=float("nan")):
    return torch.full((E, d_out, d_in + pad), fill, dtype=dtype, device=DEV)[:, :, :d_in]


class Case:
    def __init__(self, seed, n, k, E, kind, d_in, d_out, gathered, pad=0, dw="bf16", small=False):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def rand(*s):
            if small:                                    # whole numbers whose sums are exact
                return torch.randint(-1, 2, s, generator=g, device=DEV).float()
            return torch.randn(*s, generator=g, device=DEV)

        ids = make_ids(seed, n, k, E, kind)
        self.ex = sorted_batch(ids, E)
        self.off = self.ex.expert_offsets.cpu().tolist()
        self.E, self.k, self.gathered, self.d_in, self.d_out = E, k, gathered, d_in, d_out
        used = self.off[-1]
        self.row = self.ex.sorted_choice[:used].long() // k if gathered else torch.arange(used, device=DEV)
        rows = n if gathered else n * k
        # rows that no routed choice names hold NaN
        self.X, self.dY = rows_of(rows, d_in, pad), rows_of(n * k, d_out, pad)
        named = torch.zeros(rows, dtype=torch.bool, device=DEV)
        named[self.row] = True
        self.X[named] = rand(int(named.sum()), d_in).to(BF)
        self.dY[:used] = rand(used, d_out).to(BF)
        self.W = matrices(E, d_out, d_in, pad)
        self.W.copy_(rand(E, d_out, d_in))
        self.Y, self.dXs = rows_of(n * k, d_out, pad, 7.0), rows_of(n * k, d_in, pad, 7.0)
        self.dW = matrices(E, d_out, d_in, pad, torch.float32 if dw == "f32" else BF)
        self.dW.copy_(rand(E, d_out, d_in))

    def forward(self, **kw):
        srg.lora_experts_gemm(self.X, self.ex, self.W, self.Y, gathered=self.gathered, **kw)

    def backward(self, dXs=True, dW=True, **kw):
        srg.lora_experts_gemm_backward(self.dY, self.X if dW else None, self.ex,
                                       self.W if dXs else None, self.dXs if dXs else None,
                                       self.dW if dW else None, gathered=self.gathered, **kw)

    def close(self, got, ref, mag, k, what, extra=0.0):
        half = 2.0 ** -8 if got.dtype == BF else U
        tol = (k + 8) * U * mag + (half + extra) * ref.abs()
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4])

    def check_rows(self):
        used = self.off[-1]
        assert (self.Y[used:] == 7).all() and (self.dXs[used:] == 7).all()
        for e in range(self.E):
            a, b = self.off[e], self.off[e + 1]
            if a == b:
                continue
            X, W, dY = self.X[self.row[a:b]].double(), self.W[e].double(), self.dY[a:b].double()
            self.close(self.Y[a:b], X @ W.t(), X.abs() @ W.abs().t(), self.d_in, ("Y", e))
            self.close(self.dXs[a:b], dY @ W, dY.abs() @ W.abs(), self.d_out, ("dXs", e))

    def check_weights(self, old, acc):
        for e in range(self.E):
            a, b = self.off[e], self.off[e + 1]
            X, dY = self.X[self.row[a:b]].double(), self.dY[a:b].double()
            ref = dY.t() @ X + (old[e].double() if acc else 0)
            self.close(self.dW[e], ref, dY.abs().t() @ X.abs() + (old[e].double().abs() if acc else 0),
                       b - a, ("dW", e), U)


SHAPES = [
    # n, k, E, kind, d_in, d_out, gathered, pad
    (1, 1, 1, "uniform", 8, 8, True, 0),
    (1, 4, 3, "uniform", 64, 128, True, 0),
    (3, 2, 5, "bad", 136, 264, False, 8),
    (64, 8, 128, "skewed", 256, 192, True, 0),
    (100, 3, 7, "bad", 72, 520, True, 16),
    (33, 2, 1, "one", 1032, 40, False, 0),
    (50, 2, 4, "none", 64, 64, True, 0),
    (257, 1, 2, "skewed", 320, 264, True, 0),
    (700, 2, 3, "uniform", 584, 776, True, 8),
    (600, 3, 4, "skewed", 256, 512, False, 0),
    (2000, 5, 37, "skewed", 128, 136, True, 0),
    (1500, 8, 1024, "skewed", 64, 72, True, 0),
    (1024, 1, 2, "one", 512, 256, True, 8),
    (40, 4, 16, "skewed", 1032, 2056, True, 0),
    (260, 8, 16, "bad", 264, 1544, True, 8),
    (1100, 4, 8, "uniform", 520, 1032, False, 0),
    (3000, 2, 12, "bad", 320, 776, True, 0),
    (6000, 4, 8, "skewed", 584, 2056, True, 8),
    (7000, 4, 8, "bad", 2048, 1024, False, 0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "_".join(str(v) for v in s[:6]))
def test_products(shape):
    say("products", shape)
    c = Case(3, *shape)
    c.forward()
    c.backward(dW=False)
    c.check_rows()


@pytest.mark.parametrize("dw,acc", [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "_".join(str(v) for v in s[:6]))
def test_weights(shape, dw, acc):
    say("weights", shape, dw, acc)
    c = Case(4, *shape, dw=dw)
    if not acc:
        c.dW.fill_(float("nan"))
    old = c.dW.clone()
    c.backward(dXs=False, accumulate=acc)
    c.check_weights(old, acc)


def test_both_at_once_and_streams():
    c = Case(5, 300, 2, 4, "skewed", 264, 136, True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.forward(stream=side)
    c.backward(stream=side)
    torch.cuda.synchronize()
    c.check_rows()
    c.check_weights(c.dW, False)


def test_two_streams_at_once():
    a, b = Case(6, 900, 2, 5, "skewed", 520, 264, True), Case(7, 800, 3, 6, "uniform", 264, 520, False)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for c, st in ((a, s), (b, t)):
            c.forward(stream=st)
            c.backward(stream=st)
    torch.cuda.synchronize()
    for c in (a, b):
        c.check_rows()
        c.check_weights(c.dW, False)


def test_no_tokens():
    ex = srg.Experts(0, 2, 3, DEV)
    srg.lora_experts_sort(torch.empty((0, 2), dtype=torch.int32, device=DEV), ex)
    z = dict(dtype=BF, device=DEV)
    W, dW = torch.ones((3, 72, 64), **z), torch.ones((3, 72, 64), **z)
    X, Y = torch.empty((0, 64), **z), torch.empty((0, 72), **z)
    srg.lora_experts_gemm(X, ex, W, Y)
    srg.lora_experts_gemm_backward(Y, X, ex, W, torch.empty((0, 64), **z), dW, accumulate=True)
    assert (dW == 1).all()
    srg.lora_experts_gemm_backward(Y, X, ex, W, torch.empty((0, 64), **z), dW)
    assert (dW == 0).all()


def test_captured():
    """Sort, product and gradients replayed on other routings and rows."""
    n, k, E, d_in, d_out = 400, 3, 6, 136, 200
    c = Case(8, n, k, E, "uniform", d_in, d_out, True)
    ids = torch.zeros((n, k), dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        srg.lora_experts_sort(ids, c.ex)
        c.forward()
        c.backward()
    for seed, kind in ((1, "skewed"), (2, "bad"), (3, "none"), (4, "one")):
        ids.copy_(torch.from_numpy(make_ids(seed, n, k, E, kind)))
        c.X.copy_(torch.randn(n, d_in, device=DEV))
        c.dY.copy_(torch.randn(n * k, d_out, device=DEV))
        c.Y.fill_(7)
        c.dXs.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        c.off = c.ex.expert_offsets.cpu().tolist()
        c.row = c.ex.sorted_choice[:c.off[-1]].long() // k
        c.check_rows()
        c.check_weights(c.dW, False)


@pytest.mark.parametrize("n,gathered", [(40, True), (500, False)])
def test_against_differences(n, gathered):
    """<dY, Y> is linear in W and in X on their own: on whole numbers whose sums the
    types hold, differences of it are the gradients' products exactly."""
    c = Case(9, n, 2, 3, "bad", 24, 40, gathered, dw="f32", small=True)
    c.backward()
    used = c.off[-1]
    g = torch.Generator(device=DEV).manual_seed(10)

    def loss():
        c.forward()
        return float((c.Y[:used].double() * c.dY[:used].double()).sum())

    D = torch.randint(-1, 2, c.W.shape, generator=g, device=DEV).to(BF)
    W = c.W.clone()
    c.W.copy_(W + D)
    up = loss()
    c.W.copy_(W - D)
    assert up - loss() == 2 * float((c.dW.double() * D.double()).sum())
    c.W.copy_(W)
    X = c.X.clone()
    D = torch.randint(-1, 2, X.shape, generator=g, device=DEV).to(BF)
    c.X.copy_(X + D)
    up = loss()
    c.X.copy_(X - D)
    dot = float((c.dXs[:used].double() * D[c.row].double()).sum())
    assert up - loss() == 2 * dot and dot != 0


def test_rows_past_4_gib():
    """Rows whose offsets pass 2^32 bytes, on both kernels' sides of every operand."""
    n, d_in, d_out, E = 300000, 8192, 64, 3
    ids = torch.zeros((n, 1), dtype=torch.int32)
    ids[-500:] = 1
    ids[-30:] = 2
    ex = srg.Experts(n, 1, E, DEV)
    srg.lora_experts_sort(ids.to(DEV), ex)
    g = torch.Generator(device=DEV).manual_seed(11)
    X = torch.zeros((n, d_in), dtype=BF, device=DEV)
    X[-500:] = torch.randn(500, d_in, generator=g, device=DEV).to(BF)
    W = torch.randn(E, d_out, d_in, generator=g, device=DEV).to(BF)
    Y = torch.empty((n, d_out), dtype=BF, device=DEV)
    srg.lora_experts_gemm(X, ex, W, Y)
    dY = torch.randn(n, d_out, generator=g, device=DEV).to(BF)
    dXs, dW = torch.empty_like(X), torch.empty((E, d_out, d_in), dtype=torch.float32, device=DEV)
    srg.lora_experts_gemm_backward(dY, X, ex, W, dXs, dW)
    for e, (a, b) in ((1, (n - 500, n - 30)), (2, (n - 30, n))):
        x, w, y = X[a:b].double(), W[e].double(), dY[a:b].double()
        for got, ref, mag, k in ((Y[a:b], x @ w.t(), x.abs() @ w.abs().t(), d_in),
                                 (dXs[a:b], y @ w, y.abs() @ w.abs(), d_out),
                                 (dW[e], y.t() @ x, y.abs().t() @ x.abs(), b - a)):
            half = 2.0 ** -8 if got.dtype == BF else U
            assert ((got.double() - ref).abs() <= (k + 8) * U * mag + half * ref.abs()).all()
    assert not Y[:1000].any() and not dW[0].any()
