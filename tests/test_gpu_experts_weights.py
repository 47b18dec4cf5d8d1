"""Weights' gradients of experts on both of their kernel's tiles, with rows gathered and in
sorted order, for segments of many stages of 64 rows whose tiles follow each other in a
workgroup.  Tolerances as in test_gpu_experts_gemm."""
import pytest
import torch

from gpu_harness import say
from test_gpu_experts_gemm import Case

pytestmark = pytest.mark.gpu

SHAPES = [
    # n, k, E, kind, d_in, d_out, gathered, pad
    (1500, 2, 8, "uniform", 2056, 1032, True, 8),
    (1500, 2, 8, "skewed", 2056, 1032, False, 0),
    (900, 3, 8, "bad", 1288, 1800, False, 8),
    (900, 3, 8, "bad", 1288, 1800, True, 0),
    (40, 4, 16, "skewed", 1032, 2056, False, 8),
    (2500, 1, 3, "skewed", 2312, 7944, True, 0),
    (600, 3, 4, "bad", 392, 520, True, 8),
    (1100, 2, 3, "skewed", 520, 776, False, 0),
    (1700, 2, 16, "uniform", 1000, 1016, True, 0),
    (2600, 2, 16, "bad", 1000, 1016, False, 8),
]


@pytest.mark.parametrize("dw,acc", [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "_".join(str(v) for v in s[:7]))
def test_weights(shape, dw, acc):
    say("weights", shape, dw, acc)
    c = Case(31, *shape, dw=dw)
    if not acc:
        c.dW.fill_(float("nan"))
    old = c.dW.clone()
    c.backward(dXs=False, accumulate=acc)
    c.check_weights(old, acc)


@pytest.mark.parametrize("shape", SHAPES[:2], ids=lambda s: "_".join(str(v) for v in s[:7]))
def test_captured(shape):
    """Replays with other rows and the program's own work between them."""
    c = Case(32, *shape)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.backward(dXs=False)
    used = c.off[-1]
    for _ in range(3):
        c.dY[:used] = torch.randn(used, c.d_out, device=c.dY.device).to(c.dY.dtype)
        c.dW.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check_weights(c.dW, False)
        got = c.dW.clone()
        c.backward(dXs=False)
        assert torch.equal(got, c.dW)
