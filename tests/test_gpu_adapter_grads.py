"""Gradients of the multi-LoRA layer against float64.

Tolerances: a sum of k products in fp32 is off by at most (k + 8) u times the sum
of the products' magnitudes, u = 2^-24, in any order; in bf16 pools H and dH are three
bf16 whose sum they are, three products for one, each smaller by 2^-8; dX's are two,
which leave at most 2^-17 (half a step of the remainder's 8 bits, 2^-9 2^-8), and a
bf16 dX is rounded once, by at most 2^-8.  dA is held against
the dH that the call returned, and dH against float64 by itself."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def padded(rows, width, dtype, pad):
    """A row-major tensor whose rows are `pad` elements further apart, NaN between."""
    return torch.full((rows, width + pad), float("nan"), dtype=dtype, device=DEV)[:, :width]


class Case:
    def __init__(self, seed, lengths, d_in, d_out, r_max, dtype, base=3, ranks=None, pad=0,
                 shuffle=True, idle=2):
        """Slots with the given numbers of rows, `idle` slots without any, `base` rows
        without an adapter."""
        g = torch.Generator().manual_seed(seed)
        S = len(lengths) + idle
        slot = torch.cat([torch.full((k,), a) for a, k in enumerate(lengths)] +
                         [torch.full((base,), -1)]).int()
        if shuffle:
            slot = slot[torch.randperm(slot.numel(), generator=g)]
        dt = DT[dtype]
        n = slot.numel()
        self.n, self.S, self.r, self.d_in, self.d_out, self.dt = n, S, r_max, d_in, d_out, dt
        self.slot = slot.to(DEV)
        rank = torch.randint(1, r_max + 1, (S,), generator=g) if ranks is None else torch.tensor(ranks)
        self.rank = rank.int().to(DEV)

        def rand(*s):
            return torch.randn(*s, generator=g)

        self.A, self.Bt = rand(S, r_max, d_in).to(dt).to(DEV), rand(S, r_max, d_out).to(dt).to(DEV)
        self.X, self.dY = padded(n, d_in, dt, pad), padded(n, d_out, dt, pad)
        self.X.copy_(rand(n, d_in))
        self.dY.copy_(rand(n, d_out))
        self.Wt = padded(d_in, d_out, dt, pad)
        self.Wt.copy_(rand(d_in, d_out))
        self.W = self.Wt.t().contiguous()
        self.pool = srg.Pool(self.A, self.Bt, self.rank, 8.0)
        self.seg = srg.Segments(n, S, DEV)
        # (entries past a row's rank are never read as numbers)
        self.H = torch.full((n, r_max), float("nan"), device=DEV)
        srg.lora_build_shrink(self.slot, self.X, self.pool, self.seg, self.H)
        self.dH = torch.full((n, r_max), float("nan"), device=DEV)
        self.dA = torch.randn(S, r_max, d_in, generator=g).to(DEV)
        self.dBt = torch.randn(S, r_max, d_out, generator=g).to(DEV)
        self.dX = padded(n, d_in, dt, pad)

    def call(self, dX=True, dA=True, dBt=True, **kw):
        srg.lora_linear_backward(self.dY, self.Wt if dX else None, self.X if dA else None,
                                 self.H if dBt else None, self.seg, self.pool, self.dH,
                                 self.dX if dX else None, self.dA if dA else None,
                                 self.dBt if dBt else None, **kw)

    def check(self, old_a, old_b, acc=False, dX=True, dA=True, dBt=True):
        torch.cuda.synchronize()
        slot, rank = self.slot.cpu().numpy(), self.rank.cpu().numpy()
        X, dY, A, Bt = f64(self.X), f64(self.dY), f64(self.A), f64(self.Bt)
        dH, H = f64(self.dH), f64(self.H)
        split = 2.0 ** -17 if self.dt == torch.bfloat16 else 0.0
        want_a, want_b = f64(old_a), f64(old_b)
        tol_a, tol_b = np.zeros_like(want_a), np.zeros_like(want_b)
        Wt = f64(self.Wt)
        out = dY @ Wt.T
        mag = np.abs(dY) @ np.abs(Wt.T)
        for a in range(self.S):
            rows, k = np.nonzero(slot == a)[0], int(rank[a])
            if not len(rows) or not k:
                continue
            s = 8.0 / k
            ref = dY[rows] @ Bt[a, :k].T
            err = (self.d_out + 8) * U * (np.abs(dY[rows]) @ np.abs(Bt[a, :k].T))
            assert (np.abs(dH[rows, :k] - ref) <= err).all(), a
            assert np.isnan(dH[rows, k:]).all(), a
            for V, Z, want, tol in ((dH, X, want_a, tol_a), (H, dY, want_b, tol_b)):
                new = s * V[rows, :k].T @ Z[rows]
                size = s * np.abs(V[rows, :k]).T @ np.abs(Z[rows])
                want[a, :k] = new + (want[a, :k] if acc else 0)
                tol[a, :k] = (3 * len(rows) + 10) * U * size + 2 * U * np.abs(want[a, :k])
            out[rows] += s * dH[rows, :k] @ A[a, :k]
            mag[rows] += s * np.abs(dH[rows, :k]) @ np.abs(A[a, :k])
        others = [i for i in range(self.n) if slot[i] < 0 or slot[i] >= self.S or rank[slot[i]] == 0]
        assert np.isnan(dH[others]).all()
        if dA:
            assert (np.abs(f64(self.dA) - want_a) <= tol_a).all(), np.max(np.abs(f64(self.dA) - want_a) - tol_a)
        if dBt:
            assert (np.abs(f64(self.dBt) - want_b) <= tol_b).all(), np.max(np.abs(f64(self.dBt) - want_b) - tol_b)
        if dX:
            tol = (split + (self.d_out + self.r + 8) * U) * mag
            if self.dt == torch.bfloat16:
                tol = tol + 2.0 ** -8 * np.abs(out)
            assert (np.abs(f64(self.dX) - out) <= tol).all(), np.max(np.abs(f64(self.dX) - out) - tol)


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 129, 200]
CASES = {
    "ranks": dict(seed=1, lengths=LENGTHS, d_in=264, d_out=136, r_max=64, dtype="bf16"),
    "narrow": dict(seed=2, lengths=LENGTHS, d_in=8, d_out=2056, r_max=32, dtype="bf16", pad=8),
    "one_row": dict(seed=3, lengths=[1], d_in=520, d_out=1032, r_max=16, dtype="bf16", base=0, idle=0),
    "base_only": dict(seed=4, lengths=[0], d_in=64, d_out=64, r_max=8, dtype="bf16", base=5),
    "whole_ranks": dict(seed=5, lengths=[40, 3, 16, 7], d_in=1024, d_out=768, r_max=64, dtype="bf16",
                        ranks=[64, 32, 33, 0, 64, 64], pad=24),
    "f32": dict(seed=6, lengths=LENGTHS, d_in=136, d_out=264, r_max=64, dtype="f32", pad=8),
    "f32_small": dict(seed=7, lengths=[1, 5, 40], d_in=8, d_out=24, r_max=8, dtype="f32"),
    "many_slots": dict(seed=8, lengths=[1, 2, 3] * 100, d_in=256, d_out=512, r_max=16, dtype="bf16"),
    "long": dict(seed=9, lengths=[2300, 17], d_in=512, d_out=256, r_max=64, dtype="bf16", shuffle=False),
}


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_gradients(name, acc):
    c = Case(**CASES[name])
    old = c.dA.clone(), c.dBt.clone()
    c.call(accumulate=acc)
    c.check(*old, acc=acc)


@pytest.mark.parametrize("dX,dA,dBt", [(True, False, False), (False, True, False),
                                       (False, False, True), (False, False, False)])
def test_parts(dX, dA, dBt):
    c = Case(**CASES["ranks"])
    old = c.dA.clone(), c.dBt.clone()
    c.call(dX, dA, dBt)
    c.check(*old, dX=dX, dA=dA, dBt=dBt)
    assert dA or torch.equal(c.dA, old[0])
    assert dBt or torch.equal(c.dBt, old[1])


@pytest.mark.parametrize("policy", ["two_buckets", "padded"])
@pytest.mark.parametrize("name", ["ranks", "f32"])
def test_rank_policies(name, policy):
    """What lies past a row's rank, in H, dH, A and Bt, is not used as a number."""
    c = Case(**CASES[name])
    for a, k in enumerate(c.rank.tolist()):
        c.A[a, k:] = float("nan")
        c.Bt[a, k:] = float("nan")
    c.pool.set_policy(policy)
    old = c.dA.clone(), c.dBt.clone()
    c.call()
    c.check(*old)


def test_bad_slots_and_no_rows():
    c = Case(**CASES["ranks"])
    c.slot[::7] = 1000                                   # demoted to base-only
    srg.lora_build_shrink(c.slot, c.X, c.pool, c.seg, c.H)
    old = c.dA.clone(), c.dBt.clone()
    c.call()
    c.check(*old)
    seg, e = srg.Segments(0, c.S, DEV), torch.empty
    z = dict(dtype=c.dt, device=DEV)
    srg.lora_build_segments(e(0, dtype=torch.int32, device=DEV), c.pool, seg)
    before = c.dA.clone()
    srg.lora_linear_backward(e(0, c.d_out, **z), c.Wt, e(0, c.d_in, **z), e(0, c.r, device=DEV), seg,
                             c.pool, e(0, c.r, device=DEV), e(0, c.d_in, **z), c.dA, c.dBt)
    assert torch.equal(c.dA, before)


def test_an_infinity_stays_in_its_slot():
    c = Case(seed=11, lengths=[17, 33, 16], d_in=256, d_out=256, r_max=32, dtype="bf16", base=0, idle=0)
    slot = c.slot.cpu()
    last = int((slot == 0).nonzero()[-1])
    c.X[last, 5] = float("inf")
    c.dY[last, 9] = float("nan")
    c.call()
    for a in (1, 2):
        k = int(c.rank[a])
        assert torch.isfinite(c.dA[a, :k]).all() and torch.isfinite(c.dBt[a, :k]).all()
    k = int(c.rank[0])
    assert not torch.isfinite(c.dBt[0, :k, 9]).any() and torch.isfinite(c.dBt[0, :k, 8]).all()
    assert not torch.isfinite(c.dA[0, :k, 5]).any()


def test_captured_and_other_stream():
    c, e = Case(**CASES["whole_ranks"]), Case(**CASES["whole_ranks"])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        srg.lora_build_segments(c.slot, c.pool, c.seg)
        c.call(accumulate=True)
    for _ in range(3):
        new = torch.randn(c.dY.shape, device=DEV)
        c.dY.copy_(new)
        e.dY.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        e.call(accumulate=True, stream=side)
        torch.cuda.synchronize()
        for x, y in ((c.dA, e.dA), (c.dBt, e.dBt), (c.dX, e.dX)):
            assert torch.equal(x, y)


def test_against_differences():
    """The loss <Y, dY> is linear in A and in B on their own, so its difference
    between A + D and A - D is twice <dA, D>, up to the forward pass's roundings:
    (d_in + r + 8) u of the products' magnitudes for each output."""
    c = Case(seed=12, lengths=[5, 40, 17], d_in=64, d_out=96, r_max=16, dtype="f32", base=2, ranks=[16, 5, 8, 1, 1])
    c.dA.zero_()
    c.dBt.zero_()
    c.call()
    g = torch.Generator().manual_seed(13)
    slot, rank = c.slot.cpu().numpy(), c.rank.cpu().numpy()

    def loss(A, Bt):
        pool = srg.Pool(A.contiguous(), Bt.contiguous(), c.rank, 8.0)
        H, Y = torch.zeros_like(c.H), torch.empty(c.n, c.d_out, device=DEV)
        srg.lora_build_shrink(c.slot, c.X, pool, c.seg, H)
        srg.lora_linear_fused(c.X, c.W, H, c.seg, pool, Y)
        mag = np.abs(f64(c.X)) @ np.abs(f64(c.W)).T
        for a in range(c.S):
            rows, k = slot == a, rank[a]
            mag[rows] += 8.0 / k * (np.abs(f64(c.X)[rows]) @ np.abs(f64(A)[a, :k]).T) @ np.abs(f64(Bt)[a, :k])
        err = (c.d_in + c.r + 8) * U * np.sum(mag * np.abs(f64(c.dY)))
        return np.sum(f64(Y) * f64(c.dY)), err

    live = (torch.arange(c.r, device=DEV) < c.rank.unsqueeze(1)).unsqueeze(-1)
    for _ in range(3):
        D = torch.where(live, torch.randn(c.A.shape, generator=g).to(DEV), 0)
        (up, e1), (down, e2) = loss(c.A + D, c.Bt), loss(c.A - D, c.Bt)
        dot = np.sum(f64(c.dA) * f64(D))
        assert abs(up - down - 2 * dot) <= e1 + e2 + 1e-4 * np.sum(np.abs(f64(c.dA) * f64(D)))
        assert abs(dot) > 3 * (e1 + e2)                  # the difference says something
        D = torch.where(live, torch.randn(c.Bt.shape, generator=g).to(DEV), 0)
        (up, e1), (down, e2) = loss(c.A, c.Bt + D), loss(c.A, c.Bt - D)
        dot = np.sum(f64(c.dBt) * f64(D))
        assert abs(up - down - 2 * dot) <= e1 + e2 + 1e-4 * np.sum(np.abs(f64(c.dBt) * f64(D)))


# rows and ranks of every workgroup shape of dH's kernel, rows that are no multiple of its blocks
DH_CASES = [(1000, 16), (3301, 16), (1801, 32), (3301, 32), (1100, 64), (5003, 64), (16403, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d_out", [8, 264, 2056])
@pytest.mark.parametrize("n,r_max", DH_CASES)
def test_dh_of_long_batches(n, r_max, d_out, dtype):
    lengths = [n // 2, n // 4, 1, 17, 33, 64, 65, n // 16]
    lengths.append(n - sum(lengths) - 2)
    c = Case(seed=14, lengths=lengths, d_in=8, d_out=d_out, r_max=r_max, dtype=dtype, base=2, pad=8)
    old = c.dA.clone(), c.dBt.clone()
    c.call(dX=False, dA=False, dBt=False)
    c.check(*old, dX=False, dA=False, dBt=False)
