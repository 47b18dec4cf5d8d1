"""Gradients of the layer where rows, or the gradients of slots, lie more than 4 GiB from the
first.  Tolerances as in test_gpu_adapter_grads: (k + 8) u of the products' magnitudes for a
sum of k, three times the terms where H or dH enters as three bf16, 2^-17 of dX's low-rank
term (two bf16) and half a step of a bf16 result."""
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg
from gpu_harness import DEV, say

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16
ALPHA = 8.0


def within(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() - tol).max()))


def check_slot(a, k, rows, X, dY, H, dH, A, Bt, dA, dBt, old=0.0):
    """Slot a's gradients and its rows' dH; rows: their indexes."""
    s = ALPHA / k
    x, y, h, dh = X[rows].double(), dY[rows].double(), H[rows, :k].double(), dH[rows, :k].double()
    b = Bt[a, :k].double()
    within(dH[rows, :k], y @ b.t(), (y.shape[1] + 8) * U * (y.abs() @ b.abs().t()), ("dH", a))
    for v, z, got, what in ((dh, x, dA, "dA"), (h, y, dBt, "dBt")):
        ref = s * v.t() @ z + old
        size = s * v.abs().t() @ z.abs()
        within(got[a, :k], ref, (3 * len(rows) + 10) * U * size + 2 * U * ref.abs(), (what, a))


@pytest.mark.parametrize("wide", ["d_in", "d_out"])
def test_rows_past_4_gib(wide):
    say("rows", wide)
    n, r = 300000, 16
    d_in, d_out = (8192, 64) if wide == "d_in" else (64, 8192)
    g = torch.Generator(device=DEV).manual_seed(41)

    def rand(*s):
        return torch.randn(*s, generator=g, device=DEV).to(BF)

    counts = [400, 293, 7]
    slot = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    slot[-700:] = torch.repeat_interleave(torch.arange(3), torch.tensor(counts))[torch.randperm(
        700, generator=torch.Generator().manual_seed(42))].int().to(DEV)
    rank = torch.tensor([16, 5, 8, 16], dtype=torch.int32, device=DEV)
    A, Bt = rand(4, r, d_in), rand(4, r, d_out)
    X, dY = (torch.zeros((n, d), dtype=BF, device=DEV) for d in (d_in, d_out))
    X[-700:], dY[-700:] = rand(700, d_in), rand(700, d_out)
    dY[:100] = rand(100, d_out)
    Wt = rand(d_in, d_out)
    pool, seg = srg.Pool(A, Bt, rank, ALPHA), srg.Segments(n, 4, DEV)
    H, dH = (torch.full((n, r), float("nan"), device=DEV) for _ in range(2))
    srg.lora_build_shrink(slot, X, pool, seg, H)
    dX = torch.full((n, d_in), float("nan"), dtype=BF, device=DEV)
    dA, dBt = (torch.full((4, r, d), 3.0, device=DEV) for d in (d_in, d_out))
    srg.lora_linear_backward(dY, Wt, X, H, seg, pool, dH, dX, dA, dBt)
    for a in range(3):
        rows = (slot == a).nonzero().squeeze(1)
        assert len(rows) == counts[a]
        check_slot(a, int(rank[a]), rows, X, dY, H, dH, A, Bt, dA, dBt)
        assert (dA[a, int(rank[a]):] == 3).all() and (dBt[a, int(rank[a]):] == 3).all()
    assert (dA[3] == 3).all() and (dBt[3] == 3).all()
    assert torch.isnan(dH[:-700]).all() and not dX[100:-700].any()
    rows = torch.cat([torch.arange(100), torch.arange(n - 700, n)]).to(DEV)
    y, w = dY[rows].double(), Wt.double()
    ref, mag = y @ w.t(), y.abs() @ w.abs().t()
    for i, a in enumerate(slot[rows].tolist()):
        if a < 0:
            continue
        k = int(rank[a])
        s, dh = ALPHA / k, dH[rows[i], :k].double()
        ref[i] += s * dh @ A[a, :k].double()
        mag[i] += s * dh.abs() @ A[a, :k].double().abs()
    within(dX[rows], ref, (2.0 ** -17 + (d_out + r + 8) * U) * mag + HALF * ref.abs(), "dX")


@pytest.mark.parametrize("wide", ["dA", "dBt"])
def test_gradients_past_4_gib(wide):
    say("gradients", wide)
    S, r = 1100, 64
    d_in, d_out = (16384, 64) if wide == "dA" else (64, 16384)
    g = torch.Generator(device=DEV).manual_seed(43)

    def rand(*s):
        return torch.randn(*s, generator=g, device=DEV).to(BF)

    counts = {0: 5, 500: 40, 1098: 3, 1099: 77}
    slot = torch.tensor([a for a, c in counts.items() for _ in range(c)], dtype=torch.int32)
    slot = slot[torch.randperm(len(slot), generator=torch.Generator().manual_seed(44))].to(DEV)
    n = len(slot)
    A, Bt = (torch.zeros((S, r, d), dtype=BF, device=DEV) for d in (d_in, d_out))
    rank = torch.full((S,), 64, dtype=torch.int32, device=DEV)
    rank[1098] = 33
    for a in counts:
        A[a], Bt[a] = rand(r, d_in), rand(r, d_out)
    X, dY, Wt = rand(n, d_in), rand(n, d_out), rand(d_in, d_out)
    pool, seg = srg.Pool(A, Bt, rank, ALPHA), srg.Segments(n, S, DEV)
    H, dH = (torch.full((n, r), float("nan"), device=DEV) for _ in range(2))
    srg.lora_build_shrink(slot, X, pool, seg, H)
    dX = torch.empty((n, d_in), dtype=BF, device=DEV)
    dA, dBt = (torch.full((S, r, d), 3.0, device=DEV) for d in (d_in, d_out))
    srg.lora_linear_backward(dY, Wt, X, H, seg, pool, dH, dX, dA, dBt, accumulate=True)
    y, w = dY.double(), Wt.double()
    ref, mag = y @ w.t(), y.abs() @ w.abs().t()
    for a in counts:
        k, rows = int(rank[a]), (slot == a).nonzero().squeeze(1)
        check_slot(a, k, rows, X, dY, H, dH, A, Bt, dA, dBt, old=3.0)
        s, dh = ALPHA / k, dH[rows, :k].double()
        ref[rows] += s * dh @ A[a, :k].double()
        mag[rows] += s * dh.abs() @ A[a, :k].double().abs()
    within(dX, ref, (2.0 ** -17 + (d_out + r + 8) * U) * mag + HALF * ref.abs(), "dX")
    for a in (1, 499, 501, 1024, 1097):
        assert (dA[a] == 3).all() and (dBt[a] == 3).all(), a
    assert (dA[1098, 33:] == 3).all() and (dBt[1098, 33:] == 3).all()
