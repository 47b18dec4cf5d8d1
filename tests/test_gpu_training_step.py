"""The training calls together: a projection with adapters, then experts, forward and
backward, and an optimizer step of both, against float64 autograd.

Tolerances: every stage rounds its bf16 output once (2^-8 of the value) and its fp32
sum of k products by (k + 8) u of their magnitudes, u = 2^-24; the low-rank term's H is
split into two bf16 (2^-17, taken twice).  `Step.reference` carries these errors through
the stages behind them by the magnitudes of the same products.  The first step of AdamW
is w - lr wd w - lr g / (|g| + eps): its slope in g is at most lr / eps."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, HALF = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
LR, EPS, WD, ALPHA = 0.05, 0.5, 0.01, 8.0


def f64(t):
    return t.detach().double().cpu()


class Step:
    """d_in -> d_mid (adapters on a frozen weight) -> experts -> d_out."""

    def __init__(self, seed, n=96, d_in=64, d_mid=104, d_out=72, r=16, S=5, E=6, top_k=2,
                 policy="exact", bits=32):
        g = self.g = torch.Generator().manual_seed(seed)
        self.n, self.d_in, self.d_mid, self.d_out, self.r = n, d_in, d_mid, d_out, r
        self.S, self.E, self.k = S, E, top_k

        def rand(*s, dtype=BF, by=1.0):
            return (torch.randn(*s, generator=g) * by).to(dtype).to(DEV)

        ranks = torch.tensor([r, 1, r // 2, 3, r][:S])
        A, Bt = rand(S, r, d_in, by=0.2), rand(S, r, d_mid, by=0.2)
        for a in range(S):
            A[a, ranks[a]:], Bt[a, ranks[a]:] = 0, 0
        self.base = rand(d_mid, d_in, by=0.2)
        self.base_t = self.base.t().contiguous()
        self.ranks = ranks
        self.pool = srg.Pool(A, Bt, ranks.int(), ALPHA, policy)
        self.W = rand(E, d_out, d_mid, by=0.2)
        self.seg = srg.Segments(n, S, DEV)
        self.ex = srg.Experts(n, top_k, E, DEV)
        e = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=DEV)
        c = n * top_k
        self.X, self.dZ, self.route = e(n, d_in), e(n, d_out), e(n, top_k, dtype=F32)
        self.slot, self.ids = e(n, dtype=torch.int32), e(n, top_k, dtype=torch.int32)
        self.active = e(2 * S, dtype=torch.int32)
        self.H, self.dH = e(n, r, dtype=F32), e(n, r, dtype=F32)
        self.h, self.Ys, self.Z = e(n, d_mid), e(c, d_out), e(n, d_out)
        self.dYs, self.d_route, self.dhs = e(c, d_out), e(n, top_k, dtype=F32), e(c, d_mid)
        self.dh, self.dX = e(n, d_mid), e(n, d_in)
        self.dW = e(E, d_out, d_mid, dtype=F32)
        self.dA, self.dBt = e(S, r, d_in, dtype=F32), e(S, r, d_mid, dtype=F32)
        self.experts = srg.AdamW(list(self.W), list(self.dW), bits=bits, masters=True)
        self.adapters = srg.AdamW(list(A) + list(Bt), list(self.dA) + list(self.dBt), bits=bits)

    def batch(self, idle=2):
        """A new batch, into the buffers: slot `idle` has no rows, rows without an
        adapter, a token without experts, one that names an expert twice."""
        g, n = self.g, self.n
        self.X.copy_(torch.randn(n, self.d_in, generator=g))
        self.dZ.copy_(torch.randn(n, self.d_out, generator=g) * 0.1)
        self.route.copy_(torch.rand(n, self.k, generator=g))
        slot = torch.randint(-1, self.S, (n,), generator=g)
        slot[slot == idle] = -1
        ids = torch.randint(-1, self.E - 1, (n, self.k), generator=g)      # (the last: no rows)
        ids[3], ids[5] = -1, 2
        self.slot.copy_(slot)
        self.ids.copy_(ids)
        has = torch.zeros(self.S, dtype=torch.int32)
        has[slot[slot >= 0].unique()] = 1
        self.active.copy_(torch.cat([has, has]))

    def forward(self, s=None):
        srg.lora_build_shrink(self.slot, self.X, self.pool, self.seg, self.H, stream=s)
        srg.lora_linear_fused(self.X, self.base, self.H, self.seg, self.pool, self.h, stream=s)
        srg.lora_experts_sort(self.ids, self.ex, stream=s)
        srg.lora_experts_gemm(self.h, self.ex, self.W, self.Ys, stream=s)
        srg.lora_experts_combine(self.Ys, self.route, self.ex, self.Z, stream=s)

    def backward(self, s=None, accumulate=False):
        srg.lora_experts_combine_backward(self.dZ, self.Ys, self.route, self.ex, self.dYs,
                                          self.d_route, stream=s)
        srg.lora_experts_gemm_backward(self.dYs, self.h, self.ex, self.W, self.dhs, self.dW,
                                       accumulate=accumulate, stream=s)
        srg.lora_experts_combine(self.dhs, None, self.ex, self.dh, stream=s)
        srg.lora_linear_backward(self.dh, self.base_t, self.X, self.H, self.seg, self.pool, self.dH,
                                 self.dX, self.dA, self.dBt, accumulate=accumulate, stream=s)

    def update(self, s=None, seed=0):
        kw = dict(eps=EPS, weight_decay=WD, seed=seed, stream=s)
        srg.lora_adamw_step(self.experts, LR, **kw)
        srg.lora_adamw_step(self.adapters, LR, active=self.active, **kw)
        self.pool.write_b(s)

    def everything(self):
        return [self.Z, self.dX, self.d_route, self.dA, self.dBt, self.dW, self.pool.A, self.pool.Bt,
                self.pool.B, self.W, self.experts.m, self.experts.v, self.adapters.m,
                self.adapters.v, self.experts.step, self.adapters.step] + self.experts.masters

    def reference(self):
        """Name -> (value, bound of the error), from the buffers' inputs and the weights
        as they are now: values by autograd, bounds by the stages' magnitudes."""
        leaf = lambda t: f64(t).requires_grad_()
        X, A, Bt, W, route = (leaf(t) for t in (self.X, self.pool.A, self.pool.Bt, self.W, self.route))
        base, dZ, slot, ids = f64(self.base), f64(self.dZ), self.slot.cpu(), self.ids.cpu().long()
        n, r = self.n, self.r
        scale = torch.tensor([ALPHA / k for k in self.ranks.tolist()], dtype=torch.float64)
        on = slot >= 0
        sl = slot.clamp(min=0).long()
        sc = (scale[sl] * on).unsqueeze(1)
        live = (torch.arange(r) < self.ranks[sl].unsqueeze(1)) & on.unsqueeze(1)
        Ar, Br = A[sl] * live.unsqueeze(2), Bt[sl] * live.unsqueeze(2)       # of every row

        H = (Ar @ X.unsqueeze(2)).squeeze(2)
        h = X @ base.T + sc * (H.unsqueeze(1) @ Br).squeeze(1)
        h.retain_grad()
        H.retain_grad()
        keep = (ids >= 0).unsqueeze(2)
        We = W[ids.clamp(min=0)] * keep.unsqueeze(3)                         # [n, k, out, mid]
        Y = (We @ h.reshape(n, 1, -1, 1)).squeeze(3)
        Z = (route.unsqueeze(2) * Y).sum(1)
        (Z * dZ).sum().backward()

        with torch.no_grad():
            a = torch.abs
            sumU = lambda k: (k + 8) * U
            one = lambda e, t: 1.02 * (e + HALF * a(t)) + 1e-30              # a bf16 output
            magX = a(X)
            eH = sumU(self.d_in) * (a(Ar) @ magX.unsqueeze(2)).squeeze(2)
            term = lambda v, M: (v.unsqueeze(1) @ a(M)).squeeze(1)
            eh = one(sumU(self.d_in + r) * (magX @ a(base).T + sc * term(a(H), Br))
                     + sc * term(eH + 2 * 2.0 ** -17 * a(H), Br), h)
            magh = a(h).reshape(n, 1, -1, 1)
            eY = one((a(We) @ (eh.reshape(n, 1, -1, 1) + sumU(self.d_mid) * magh)).squeeze(3), Y)
            w3 = a(route).unsqueeze(2)
            eZ = one((w3 * eY).sum(1) + sumU(self.k) * (w3 * a(Y)).sum(1), Z)
            e_route = 1.02 * ((a(dZ).unsqueeze(1) * (eY + sumU(self.d_out) * a(Y))).sum(2))
            dY = route.unsqueeze(2) * dZ.unsqueeze(1) * keep
            edY = one(2 * U * a(dY), dY)
            back = lambda v: (v.unsqueeze(2) @ a(We)).squeeze(2)
            dhs = (dY.unsqueeze(2) @ We).squeeze(2)
            edhs = one(back(edY + sumU(self.d_out) * a(dY)), dhs)
            dh = dhs.sum(1)
            edh = one(edhs.sum(1) + sumU(self.k) * a(dhs).sum(1), dh)
            eW = torch.zeros_like(W)
            for j in range(self.k):
                ok = ids[:, j] >= 0
                t = edY[:, j].unsqueeze(2) * a(h).unsqueeze(1) + a(dY[:, j]).unsqueeze(2) * \
                    (eh + sumU(n * self.k) * a(h)).unsqueeze(1)
                eW.index_add_(0, ids[ok, j], t[ok])
            dH = (Br @ dh.unsqueeze(2)).squeeze(2)                           # (without the scale)
            magdH = (a(Br) @ a(dh).unsqueeze(2)).squeeze(2)
            edH = (a(Br) @ edh.unsqueeze(2)).squeeze(2) + sumU(self.d_mid) * magdH
            eA, eB = torch.zeros_like(A), torch.zeros_like(Bt)
            s3, sumN = sc.unsqueeze(2), sumU(3 * n)
            ta = s3 * (edH + sumN * a(dH)).unsqueeze(2) * magX.unsqueeze(1)
            tb = s3 * ((eH + sumN * a(H)).unsqueeze(2) * a(dh).unsqueeze(1)
                       + a(H).unsqueeze(2) * edh.unsqueeze(1)) * live.unsqueeze(2)
            eA.index_add_(0, sl[on], ta[on])
            eB.index_add_(0, sl[on], tb[on])
            eX = one(edh @ a(base) + sumU(self.d_mid + r) * (a(dh) @ a(base) + sc * term(a(dH), Ar))
                     + sc * term(edH + 2 * 2.0 ** -17 * a(dH), Ar), X.grad)
        tiny = 1e-30
        return dict(h=(h.detach(), eh), Z=(Z.detach(), eZ), d_route=(route.grad, e_route + tiny),
                    dh=(h.grad, edh), dX=(X.grad, eX), dW=(W.grad, 1.02 * eW + tiny),
                    dA=(A.grad, 1.02 * eA + tiny), dBt=(Bt.grad, 1.02 * eB + tiny))


def within(got, want, err, what):
    over = (f64(got) - want).abs() - err
    assert (over <= 0).all(), (what, float(over.max()))


def adamw_first(w, g, eg, rounded):
    up = LR * g / (g.abs() + EPS)
    new = w - LR * WD * w - up
    err = LR / EPS * eg + U * (3 * w.abs() + 24 * up.abs())
    return new, 1.02 * (err + (HALF * new.abs() if rounded else 0)) + 1e-30


@pytest.mark.parametrize("policy", ["exact", "two_buckets", "padded"])
def test_first_step(policy):
    s = Step(1, policy=policy)
    s.batch()
    s.forward()
    s.backward()
    r = s.reference()
    for name, (want, err) in r.items():
        within(getattr(s, name), want, err, name)
        assert float(err.max()) < 0.6 * float(want.abs().max()), name        # (the bounds say something)
    A, Bt, W = f64(s.pool.A), f64(s.pool.Bt), f64(s.W)
    s.update()
    on = s.active[:s.S].bool().cpu()
    assert not on.all() and on.any()
    for w, key, got in ((A, "dA", s.pool.A), (Bt, "dBt", s.pool.Bt)):
        new, err = adamw_first(w, *r[key], True)
        within(got[on.to(DEV)], new[on], err[on], key)
        assert torch.equal(f64(got)[~on], w[~on])                            # idle: as it was
    new, err = adamw_first(W, *r["dW"], False)
    within(torch.stack(s.experts.masters), new, err, "masters")
    assert torch.equal(s.W, torch.stack(s.experts.masters).to(BF))
    assert torch.equal(s.pool.B, s.pool.Bt.transpose(1, 2))
    assert torch.equal(s.adapters.step, s.active) and (s.experts.step == 1).all()
    # the next batch sees the new weights
    s.batch(idle=0)
    s.forward()
    r = s.reference()
    within(s.h, *r["h"], "h")
    within(s.Z, *r["Z"], "Z")


def test_gradients_of_two_batches_add_up():
    s, t = Step(2), Step(2)
    s.batch()
    s.forward()
    s.backward()
    first = [x.clone() for x in (s.dA, s.dBt, s.dW)]
    one = s.reference()
    s.batch(idle=1)
    s.forward()
    s.backward(accumulate=True)
    two = s.reference()
    for got, old, key in zip((s.dA, s.dBt, s.dW), first, ("dA", "dBt", "dW")):
        (w1, e1), (w2, e2) = one[key], two[key]
        within(got, w1 + w2, e1 + e2 + 2 * U * (w1 + w2).abs(), key)
        assert not torch.equal(got, old)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_and_another_stream(bits):
    """Steps from a graph, from a stream of their own and from the current one leave
    the same bits; idle slots keep their moments."""
    c, e, o = (Step(3, bits=bits) for _ in range(3))
    side = torch.cuda.Stream()

    def run(s, stream=None):
        s.forward(stream)
        s.backward(stream)
        s.update(stream, seed=7)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(c)
    for i in range(4):
        for s in (c, e, o):
            s.batch(idle=i % c.S)
        torch.cuda.synchronize()
        graph.replay()
        run(e)
        run(o, side)
        torch.cuda.synchronize()
        for x, y, z in zip(c.everything(), e.everything(), o.everything()):
            assert torch.equal(x, y) and torch.equal(x, z)
    steps = c.adapters.step.cpu()
    assert steps.max() <= 4 and (steps[:c.S] < 4).any() and (c.experts.step == 4).all()
