"""MXFP4 calls on batches and weights past what a 16-bit grid or a 32-bit offset
holds; tolerances as in test_gpu_mxfp4_kernels.py."""
import numpy as np
import pytest
import torch

import oracle
import segmented_rank_gemm_segment_amd as srg
from gpu_harness import DEV, say
from test_gpu_mxfp4 import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    srg.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def random_mxfp4(n, d, seed, lo=118, hi=123):
    q, s = srg.mxfp4_empty(n, d, DEV)
    q.random_(0, 256, generator=gen(seed))
    s.random_(lo, hi + 1, generator=gen(seed + 1))
    return q, s


def values(q, s):
    return torch.from_numpy(oracle.decode_mxfp4(q.cpu().numpy(), s.cpu().numpy())).to(DEV)


def check(out, X64, W64, what):
    Y64 = X64 @ W64.t()
    tol = 2.0 ** -8 * Y64.abs() + 1.01 * X64.shape[1] * U * (X64.abs() @ W64.abs().t())
    assert bool(((out.double() - Y64).abs() <= tol).all()), what


@pytest.mark.parametrize("n,d", [(65535 * 64 + 77, 32), (65535 + 70, 2080)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_more_rows_than_a_grid_has(n, d, dtype):
    """Rows that repeat a block of 4099: codes, scales and values repeat with it."""
    say("rows", n, d, dtype)
    m = 4099
    X0 = torch.randn(m, d, device=DEV, generator=gen(d)).to(dtype)
    X = X0.repeat((n + m - 1) // m, 1)[:n]
    q, s = srg.mxfp4_empty(n, d, DEV)
    q.fill_(0xAB)
    s.fill_(0xCD)
    srg.lora_mxfp4_quantize(X, q, s)
    q0, s0 = oracle.quantize_mxfp4(X0[:64].double().cpu().numpy())
    assert np.array_equal(q[:64].cpu().numpy(), q0) and np.array_equal(s[:64].cpu().numpy(), s0)
    assert torch.equal(q[m:], q[:n - m]) and torch.equal(s[m:], s[:n - m])
    out = torch.full((n, d), 9.0, dtype=dtype, device=DEV)
    srg.lora_mxfp4_dequantize(q, s, out)
    assert torch.equal(out[:64].double(), torch.from_numpy(oracle.decode_mxfp4(q0, s0)).to(DEV))
    assert torch.equal(out[m:], out[:n - m])


@pytest.mark.parametrize("both", [False, True])
def test_products_past_4_gib(both):
    """530,000 rows: X in bf16 and Y pass 2^32 bytes."""
    n, d_in, d_out = 530_000, 4096, 4104
    say("far rows", both)
    Wq, ws = random_mxfp4(d_out, d_in, 1)
    X = torch.randn(n, d_in, dtype=torch.bfloat16, device=DEV, generator=gen(2))
    Y = torch.empty((n, d_out), dtype=torch.bfloat16, device=DEV)
    rows = torch.cat([torch.arange(200), torch.randint(200, n - 300, (400,), generator=torch.Generator().manual_seed(3)),
                      torch.arange(n - 300, n)]).to(DEV)
    if both:
        Xq = srg.mxfp4_empty(n, d_in, DEV)
        srg.lora_mxfp4_quantize(X, *Xq)
        srg.lora_base_gemm_mxfp4(*Xq, Wq, ws, Y)
        X64 = values(Xq[0][rows], Xq[1][rows])
    else:
        srg.lora_base_gemm_mxfp4w(X, Wq, ws, Y)
        X64 = X[rows].double()
    check(Y[rows], X64, values(Wq, ws), both)


@pytest.mark.parametrize("rows_per_expert", [2, 6, 20, 100])
def test_experts_weights_past_4_gib(rows_per_expert):
    """160 experts of 4096 -> 14336: their codes pass 2^32 bytes."""
    E, d_in, d_out = 160, 4096, 14336
    say("far experts", rows_per_expert)
    q, s = random_mxfp4(E * d_out, d_in, 5)
    Wq, ws = q.view(E, d_out, d_in // 2), s.as_strided((E, d_out, d_in // 32), (d_out * s.stride(0), s.stride(0), 1))
    n = E * rows_per_expert
    ids = torch.randperm(n, device=DEV, generator=gen(6)).remainder(E).int().view(n, 1)
    ex = srg.Experts(n, 1, E, DEV)
    srg.lora_experts_sort(ids, ex)
    X = torch.randn(n, d_in, dtype=torch.bfloat16, device=DEV, generator=gen(7))
    Y = torch.full((n, d_out), 7.0, dtype=torch.bfloat16, device=DEV)
    srg.lora_experts_gemm_mxfp4w(X, ex, Wq, ws, Y)
    for e in (0, 1, 73, 146, 147, 159):
        p = slice(e * rows_per_expert, (e + 1) * rows_per_expert)
        check(Y[p], X[ex.sorted_choice[p].long()].double(), values(Wq[e], ws[e]), e)
