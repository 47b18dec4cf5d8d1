"""AdamW over many tensors against float64.

Tolerances, from the roundings of the fp32 arithmetic (half a step u = 2^-24
each): m' = b1 m + c1 g has at most five on each term's way (the factor, the
gradient's scale, the product, the sum), v' at most eight, all relative to terms
that do not cancel in v'.  The quotient and its factors add at most 16 to the
update, and the error of m' passes through it; w' rounds three times.  A bf16
tensor is rounded once more, by at most 2^-8.  8-bit codes are exact unless the
uniform number lies within the error of the value's place between two codes: the
place's error is that of z (at most 24 roundings) times z over the codes'
distance, which is at most 64 codes for v and 64 for m: 24 * 64 * 2^-24 < 1e-4."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg
import train_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [(1,), (7, 9), (256,), (255,), (257,), (0,), (4096,), (64, 64), (4099,), (3, 5, 1111)]


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def setup(seed, sizes, p="f32", g="f32", bits=32, masters=False, scale=1e-2):
    gen = torch.Generator().manual_seed(seed)
    params = [(torch.randn(s, generator=gen) * 0.1).to(DT[p]).to(DEV) for s in sizes]
    grads = [(torch.randn(s, generator=gen) * scale).to(DT[g]).to(DEV) for s in sizes]
    return srg.AdamW(params, grads, bits=bits, masters=masters or None), gen


def snapshot(opt):
    s = dict(step=opt.step.cpu().numpy().copy(), m=[], v=[], w=[], g=[])
    for i, p in enumerate(opt.params):
        a, n = opt.starts[i], p.numel()
        blk = slice(a // 256, (a + n + 255) // 256)
        if opt.bits == 8:
            s["m"].append(ref.value_m(opt.m[a:a + n].cpu().numpy(), opt.m_scale[blk].cpu().numpy()))
            s["v"].append(ref.value_v(opt.v[a:a + n].cpu().numpy(), opt.v_scale[blk].cpu().numpy()))
        else:
            s["m"].append(f64(opt.m[a:a + n]))
            s["v"].append(f64(opt.v[a:a + n]))
        s["w"].append(f64(opt.masters[i] if opt.masters is not None else p))
        s["g"].append(f64(opt.grads[i]))
    return s


def check(opt, before, lr, seed=0, active=None, gscale=1.0, b1=0.9, b2=0.999, eps=1e-8, wd=0.01):
    after = snapshot(opt)
    for i, p in enumerate(opt.params):
        on = active is None or active[i] != 0
        t = int(before["step"][i]) + (1 if on else 0)
        assert int(after["step"][i]) == t, i
        if not on:
            for k in ("m", "v", "w"):
                assert np.array_equal(after[k][i], before[k][i]), (i, k)
            continue
        g, w0 = before["g"][i] * gscale, before["w"][i]
        w, m, v, up = ref.adamw(w0, g, before["m"][i], before["v"][i], t, lr, b1, b2, eps, wd)
        tm = 5 * U * (np.abs(b1 * before["m"][i]) + np.abs((1 - b1) * g)) + 1e-38
        tv = 8 * U * v + 1e-38
        # (what m' is off by passes through the quotient)
        den = np.sqrt(v / (1 - b2 ** t)) + eps
        tw = U * (3 * np.abs(w0) + 16 * np.abs(up)) + lr / (1 - b1 ** t) / den * tm
        if opt.masters is None and p.dtype == torch.bfloat16:
            tw = tw + 2.0 ** -8 * np.abs(w)
        assert (np.abs(after["w"][i] - w) <= tw).all(), (i, np.max(np.abs(after["w"][i] - w) - tw))
        if opt.masters is not None:
            assert torch.equal(p, opt.masters[i].to(p.dtype)), i
        if opt.bits == 32:
            assert (np.abs(after["m"][i] - m) <= tm).all(), i
            assert (np.abs(after["v"][i] - v) <= tv).all(), i
            continue
        a, n = opt.starts[i], p.numel()
        if n == 0:
            continue
        blk = slice(a // 256, (a + n + 255) // 256)
        u = ref.uniform(seed, t, i, 0, n)
        for x, power, levels, codes, scales, floor in (
                (m, 2, 127, opt.m, opt.m_scale, 0), (v, 4, 255, opt.v, opt.v_scale, 1)):
            got = codes[a:a + n].cpu().numpy().astype(np.int64)
            at, top = ref.place(np.abs(x), power, levels)
            sc = scales[blk].cpu().numpy().astype(np.float64)
            # (m' may cancel: its error is relative to its terms)
            err = np.max(np.pad(tm if power == 2 else tv, (0, -n % 256)).reshape(-1, 256), 1)
            assert (np.abs(sc - top) <= err).all(), i
            want = np.ceil(at - u)                       # the upper code where the share is above u
            sure = np.abs(at - u - np.round(at - u)) > 1e-4
            if power == 2:                               # ... and where m' is exact enough
                t_rep = np.repeat(np.where(top > 0, top, 1), 256)[:n]
                slip = (tm + np.repeat(err, 256)[:n]) / t_rep * levels ** 2 / (2 * np.floor(at) + 1)
                sure &= np.abs(at - u - np.round(at - u)) > slip + 1e-4
            want = np.clip(np.where(x != 0, np.maximum(want, floor), 0), 0, levels)
            want = (want * np.sign(x)).astype(np.int64)
            assert sure.mean() > 0.99 or n < 4000
            assert np.array_equal(got[sure], want[sure]), (i, power, np.sum(got[sure] != want[sure]))
            assert (np.abs(got - want) <= 1).all(), (i, power)


VARIANTS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "f32", False),
            ("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g,masters", VARIANTS, ids=[f"{p}_{g}{'_w' if w else ''}" for p, g, w in VARIANTS])
def test_steps(p, g, masters, bits):
    opt, gen = setup(1, SIZES, p, g, bits, masters)
    assert opt.numel == sum(-(-q.numel() // 256) * 256 for q in opt.params)
    for k in range(3):                                   # moments of zero, then others
        before = snapshot(opt)
        srg.lora_adamw_step(opt, 1e-2, seed=77 + k)
        check(opt, before, 1e-2, seed=77 + k)
        for q in opt.grads:
            q.copy_(torch.randn(q.shape, generator=gen) * 10.0 ** -k)


@pytest.mark.parametrize("bits", [32, 8])
def test_active_scale_rate_and_stream(bits):
    opt, gen = setup(2, SIZES * 30, "bf16", "f32", bits, True)     # 300 tensors
    flags = torch.randint(0, 2, (len(opt.params),), generator=gen, dtype=torch.int32)
    lr = torch.tensor([3e-3], device=DEV)
    gs = torch.tensor([0.25], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        before = snapshot(opt)
        act = flags.to(DEV)
        torch.cuda.synchronize()
        srg.lora_adamw_step(opt, lr, 0.8, 0.95, 1e-6, 0.1, grad_scale=gs, active=act, seed=5,
                            stream=side)
        torch.cuda.synchronize()
        check(opt, before, float(lr), 5, flags.numpy(), 0.25, 0.8, 0.95, 1e-6, 0.1)


def test_far_step_counts():
    """Bias corrections of a first step and of one past 2^20."""
    opt, _ = setup(3, [(300,), (300,)])
    opt.step.copy_(torch.tensor([0, 1 << 20]))
    before = snapshot(opt)
    srg.lora_adamw_step(opt, 1e-3)
    check(opt, before, 1e-3)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps(bits):
    """A captured step replayed, with eager work between, is the eager steps."""
    a, _ = setup(4, SIZES, "bf16", "bf16", bits, True)
    b, gen = setup(4, SIZES, "bf16", "bf16", bits, True)
    lr = torch.tensor([1e-2], device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        srg.lora_adamw_step(a, lr, seed=9)
    assert int(a.step.sum()) == 0
    for k in range(4):
        for x, y in zip(a.grads, b.grads):
            x.copy_(torch.randn(x.shape, generator=gen))
            y.copy_(x)
        lr.fill_(10.0 ** -k)
        graph.replay()
        srg.lora_adamw_step(b, lr, seed=9)
        torch.cuda.synchronize()
        for name in ("m", "v", "step", "m_scale", "v_scale"):
            x, y = getattr(a, name), getattr(b, name)
            assert x is None or torch.equal(x, y), (k, name)
        for x, y in zip(a.params + a.masters, b.params + b.masters):
            assert torch.equal(x, y), k


def test_values_not_finite():
    """An infinity or NaN spoils its element with 32-bit moments, its block's
    moments with 8-bit ones, and nothing else."""
    for bits in (32, 8):
        opt, _ = setup(5, [(1024,), (512,)], bits=bits)
        opt.grads[0][300] = float("inf")
        opt.grads[0][700] = float("nan")
        srg.lora_adamw_step(opt, 1e-2)
        bad = torch.zeros(1024, dtype=torch.bool)
        bad[700] = True
        bad[300] = True                                  # inf / inf
        assert torch.equal(~torch.isfinite(opt.params[0]).cpu(), bad)
        assert torch.isfinite(opt.params[1]).all()
        if bits == 8:
            assert torch.isnan(opt.m_scale).cpu().tolist() == [False, True, True, False, False, False]
            m, v = torch.empty(opt.numel, device=DEV), torch.empty(opt.numel, device=DEV)
            srg.lora_adamw_read(opt, m, v)
            assert torch.isnan(m[256:768]).all() and torch.isnan(v[256:768]).all()
            assert torch.isfinite(m[:256]).all() and torch.isfinite(v[768:]).all()


def test_small_blocks_become_zeros():
    opt, _ = setup(6, [(256,)], bits=8)
    opt.grads[0].fill_(2.0 ** -99)
    srg.lora_adamw_step(opt, 1e-2)
    assert not opt.m.any() and not opt.v.any() and float(opt.m_scale) == float(opt.v_scale) == 0.0
    assert torch.isfinite(opt.params[0]).all()


def test_steps_of_small_scales():
    """Second moments whose scales are just above 2^-100, where a code's unit, 255^-4 of
    it, is below the smallest normal number."""
    opt, gen = setup(13, [(2048,), (300,)], bits=8)
    for step in range(3):
        for g in opt.grads:
            g.copy_((torch.rand(g.shape, generator=gen) + 0.5) * 2.0 ** -44)
        before = snapshot(opt)
        srg.lora_adamw_step(opt, 1e-2, seed=step)
        assert (opt.v_scale > 0).all() and (opt.v_scale < 2.0 ** -94).all()
        check(opt, before, 1e-2, seed=step)
    m, v = torch.empty(opt.numel, device=DEV), torch.empty(opt.numel, device=DEV)
    srg.lora_adamw_read(opt, m, v)
    want = ref.value_v(opt.v.cpu().numpy(), opt.v_scale.cpu().numpy())
    assert (np.abs(f64(v) - want) <= 4 * U * want + 2.0 ** -149).all()


def test_largest_blocks():
    """Moments up to their documented bounds keep codes in range; past them the scale is NaN."""
    opt, _ = setup(14, [(256,), (256,), (256,)], bits=8)
    kw = dict(beta1=0.0, beta2=0.999)                    # m = g, v = 0.001 g^2
    sign = torch.where(torch.arange(256, device=DEV) % 2 == 0, 1.0, -1.0)
    opt.grads[0].copy_(sign * 2.0 ** 63)                 # v just below 2^118 ...
    opt.grads[1].copy_(sign * 2.0 ** 63.99)              # ... and above
    opt.grads[2].copy_(sign * 2.0 ** 40)
    srg.lora_adamw_step(opt, 1e-2, **kw)
    assert torch.isfinite(opt.m_scale).all()
    assert torch.isfinite(opt.v_scale[[0, 2]]).all() and torch.isnan(opt.v_scale[1])
    assert (opt.m.abs() == 127).all() and torch.equal(opt.m[:256].sign().float(), sign)
    assert (opt.v[:256] == 255).all() and not opt.v[256:512].any()
    opt.m_scale[2] = 2.0 ** 126                          # m = 0.9 of 2^126, then 1.1
    opt.v.zero_()
    opt.v_scale.zero_()
    for g in opt.grads:
        g.zero_()
    srg.lora_adamw_step(opt, 1e-2, beta1=0.9)
    assert torch.isfinite(opt.m_scale).all() and (opt.m[512:].abs() == 127).all()
    opt.m_scale[2] = 2.0 ** 126 * 1.2
    srg.lora_adamw_step(opt, 1e-2, beta1=0.9)
    assert torch.isnan(opt.m_scale[2]) and not opt.m[512:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_read(dtype):
    opt, _ = setup(7, SIZES, bits=8)
    srg.lora_adamw_step(opt, 1e-2)
    m = torch.empty(opt.numel, dtype=DT[dtype], device=DEV)
    v = torch.empty_like(m)
    srg.lora_adamw_read(opt, m, v)
    tol = 4 * U + (2.0 ** -8 if dtype == "bf16" else 0.0)
    for got, want in ((m, ref.value_m(opt.m.cpu().numpy(), opt.m_scale.cpu().numpy())),
                      (v, ref.value_v(opt.v.cpu().numpy(), opt.v_scale.cpu().numpy()))):
        assert (np.abs(f64(got) - want) <= tol * np.abs(want) + 1e-37).all()


def test_rounding_is_fair():
    """The codes' values are the moments on average: the mean error of n values,
    each off by at most its codes' distance d and fair, is below five of its
    standard deviations, at most sqrt(sum d^2 / 4) / n."""
    n = 1 << 16
    opt, _ = setup(8, [(n,)], bits=8)
    srg.lora_adamw_step(opt, 1e-2, seed=3)
    g = f64(opt.grads[0])
    for x, power, levels, value in ((0.1 * g, 2, 127, ref.value_m(opt.m.cpu().numpy(), opt.m_scale.cpu().numpy())),
                                    (0.001 * g ** 2, 4, 255, ref.value_v(opt.v.cpu().numpy(), opt.v_scale.cpu().numpy()))):
        at, top = ref.place(np.abs(x), power, levels)
        c = np.floor(at)
        d = np.repeat(top, 256) * (((c + 1) / levels) ** power - (c / levels) ** power)
        # (code 0 is left out: second moments above 0 take code 1)
        use = c >= 1
        bound = 5 * np.sqrt(np.sum(d[use] ** 2) / 4)
        assert abs(np.sum((np.abs(value) - np.abs(x))[use])) <= bound + 1e-5 * np.sum(np.abs(x))


def test_same_call_same_bits():
    outs = []
    for _ in range(2):
        opt, _ = setup(9, SIZES, "bf16", "f32", 8)
        srg.lora_adamw_step(opt, 1e-2, seed=123)
        outs.append([opt.m.clone(), opt.v.clone()] + [p.clone() for p in opt.params])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_offsets_past_32_bits():
    """One tensor of more than 2^32 elements, and one behind it."""
    n = (1 << 32) + 5000
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    q, h = torch.zeros(700, device=DEV).bfloat16(), torch.full((700,), 0.5, device=DEV).bfloat16()
    gen = torch.Generator().manual_seed(10)
    parts = [(0, 4096), ((1 << 31) - 2048, 4096), ((1 << 32) - 2048, 7048)]
    for a, k in parts:
        p[a:a + k] = (torch.randn(k, generator=gen) * 0.1).to(DEV).bfloat16()
        g[a:a + k] = torch.randn(k, generator=gen).to(DEV).bfloat16()
    kept = [(f64(p[a:a + k]), f64(g[a:a + k])) for a, k in parts]
    opt = srg.AdamW([p, q], [g, h], bits=8)
    srg.lora_adamw_step(opt, 1e-2, seed=1)
    for (a, k), (w0, g0) in zip(parts, kept):
        w, m, v, up = ref.adamw(w0, g0, 0.0, 0.0, 1, 1e-2)
        assert (np.abs(f64(p[a:a + k]) - w) <= 2.0 ** -8 * np.abs(w) + 32 * U * (np.abs(w0) + np.abs(up))).all()
        u = ref.uniform(1, 1, 0, a, k)
        first = a // 256 * 256
        assert first == a
        at, _ = ref.place(v, 4, 255)
        want = np.where(v > 0, np.clip(np.ceil(at - u), 1, 255), 0)
        sure = np.abs(at - u - np.round(at - u)) > 1e-4
        got = opt.v[a:a + k].cpu().numpy()
        assert np.array_equal(got[sure], want[sure].astype(np.uint8))
    want = ref.adamw(np.zeros(700), np.full(700, 0.5), 0.0, 0.0, 1, 1e-2)[0]
    assert (np.abs(f64(q) - want) <= 2.0 ** -8 * np.abs(want) + 1e-7).all()
