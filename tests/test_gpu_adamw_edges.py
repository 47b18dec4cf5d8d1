"""AdamW at the ends of its ranges: codes next to the border between two of them, second
moments below the normal numbers, the smallest eps.

A code's place.  On a first step m' = c1 g and v' = c2 g^2 are one and two fp32 roundings,
which are repeated here, so only what the codes add is left: z = L / top x (the division and
the product: 2 roundings of half a step, u = 2^-24 each), the difference to c's own power
and the product that it is held against (at most 4 roundings of the codes' distance).  In
codes that is 2 u z / distance + 4 u: z / distance is at most 127^2 / 253 = 63.8 for m and
255^4 / (255^4 - 254^4) = 64.2 for v, together below 8e-6."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg
import train_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F = np.float32


def test_codes_beside_a_border():
    """Every element whose uniform number is further than that from its place between two
    codes has the code of the definition, and the others go up as often as down."""
    n, seed = 1 << 22, 21
    gen = torch.Generator().manual_seed(20)
    g = (0.75 + 0.25 * torch.rand(n, generator=gen)) * torch.where(torch.rand(n, generator=gen) < 0.5, -1, 1)
    g[1::2] *= 0.02 + torch.rand(n // 2, generator=gen)            # and all codes below
    opt = srg.AdamW([torch.zeros(n, device=DEV)], [g.to(DEV)], bits=8)
    srg.lora_adamw_step(opt, 1e-2, seed=seed)
    u = ref.uniform(seed, 1, 0, 0, n)
    x = g.numpy()
    m = x * F(1.0 - 0.9)
    v = (x * x) * F(256.0 * F(1.0 - 0.999))
    for what, y, power, levels, got in (("m", m, 2, 127, opt.m), ("v", v, 4, 255, opt.v)):
        at, _ = ref.place(np.abs(y).astype(np.float64), power, levels)
        off = at - u - np.round(at - u)                  # from the border
        want = np.maximum(np.ceil(at - u), 1 if power == 4 else 0)
        diff = np.abs(got.cpu().numpy().astype(np.int64)) - want
        far = np.abs(off) > 8e-6
        assert not diff[far].any(), (what, int(np.count_nonzero(diff[far])), np.abs(off[diff != 0]).max())
        up, down = np.count_nonzero(diff > 0), np.count_nonzero(diff < 0)
        # five standard deviations of a fair coin's
        assert abs(up - down) <= 5 * np.sqrt(up + down) + 1, (what, up, down)


U, HALF_STEP = 2.0 ** -24, 2.0 ** -150     # of fp32: relative, and of its subnormal numbers


@pytest.mark.parametrize("eps", [1e-20, 1e-25, 1e-30, 2.0 ** -126])
def test_second_moments_below_the_normal_numbers(eps):
    """Gradients of 1e-20 to 1e-17, whose second moments are subnormal, beside an eps that
    does not hide their roots.

    v' is off by eight roundings u of it and by half a subnormal step, h, for each of
    g^2 (then times 0.001), its product and the sum: dv <= 8 u v + 2.001 h.  Its root is off
    by dv / sqrt(v) at most, and the update by that against the denominator that is left.
    m' and w' round as usual (five u and three u of their terms, sixteen u of the update)."""
    n, lr, b1, b2, wd = 4099, 1e-2, 0.9, 0.999, 0.01
    gen = torch.Generator().manual_seed(22)
    w = (torch.randn(n, generator=gen) * 0.1).to(DEV)
    g = torch.zeros(n, device=DEV)
    opt = srg.AdamW([w], [g])
    for t in (1, 2, 3):
        size = 10.0 ** (-20 + 3 * torch.rand(n, generator=gen, dtype=torch.float64))
        g.copy_((size * torch.where(torch.rand(n, generator=gen) < 0.5, -1, 1)).float())
        f64 = lambda x: x[:n].double().cpu().numpy()
        w0, g0, m0, v0 = f64(w), f64(g), f64(opt.m), f64(opt.v)
        srg.lora_adamw_step(opt, lr, b1, b2, eps, wd)
        want, m, v, up = ref.adamw(w0, g0, m0, v0, t, lr, b1, b2, eps, wd)
        dm = 5 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g0))
        dv = 8 * U * v + 2.001 * HALF_STEP
        assert (np.abs(f64(opt.m) - m) <= dm).all() and (np.abs(f64(opt.v) - v) <= dv).all()
        left = 1 / np.sqrt(1 - b2 ** t)
        den, dden = np.sqrt(v) * left + eps, dv / np.sqrt(v) * left
        assert (dden < 0.05 * den).all()
        tol = 3 * U * np.abs(w0) + np.abs(up) * (16 * U + dden / (den - dden)) \
            + lr / (1 - b1 ** t) / (den - dden) * dm
        assert (np.abs(f64(w) - want) <= tol).all(), (t, np.max(np.abs(f64(w) - want)))


def test_smallest_eps_beside_8_bit_moments():
    """eps 2^-40 is taken: blocks of second moments that became zeros, here of gradients
    2^-48, leave m over eps and the new gradient's root, not more."""
    w, g = torch.zeros(256, device=DEV), torch.full((256,), 2.0 ** -48, device=DEV)
    opt = srg.AdamW([w], [g], bits=8)
    for t in range(1, 5):
        before = w.clone()
        srg.lora_adamw_step(opt, 1.0, eps=2.0 ** -40, weight_decay=0.0)
        assert not opt.v.any() and opt.m.any()
        # at most the step that eps alone leaves: |m| / (1 - b1^t) = 2^-48 but for the codes
        assert (before - w).abs().max() <= 2.0 ** -8 * 1.05


@pytest.mark.parametrize("p,g,masters", [(torch.float32, torch.float32, None),
                                         (torch.bfloat16, torch.bfloat16, True)])
def test_codes_between_tensors_do_not_count(p, g, masters):
    """What stands in the 8-bit moments behind a tensor's last element, in its last block,
    changes neither the block's scale nor the tensor's own codes."""
    sizes = [1, 7, 8, 9, 255, 256, 257, 4091, 5000]
    opts = []
    for _ in range(2):
        gen = torch.Generator().manual_seed(23)
        opts.append(srg.AdamW([(torch.randn(n, generator=gen) * 0.1).to(p).to(DEV) for n in sizes],
                              [torch.zeros(n, dtype=g, device=DEV) for n in sizes], bits=8,
                              masters=masters))
    a, b = opts
    inside = torch.zeros(a.numel, dtype=torch.bool, device=DEV)
    for at, n in zip(a.starts, sizes):
        inside[at:at + n] = True
    gen = torch.Generator().manual_seed(24)
    for step in range(4):
        for x, y in zip(a.grads, b.grads):
            # (small ones behind the first step, beside which a large code's value shows)
            x.copy_(torch.randn(x.shape, generator=gen) * 10.0 ** -step)
            y.copy_(x)
        b.m.masked_fill_(~inside, 127 if step % 2 else -128)
        b.v.masked_fill_(~inside, 255)
        for o in opts:
            srg.lora_adamw_step(o, 1e-2, beta1=0.5, beta2=0.9, seed=step)
        assert torch.equal(a.m_scale, b.m_scale) and torch.equal(a.v_scale, b.v_scale), step
        assert torch.equal(a.m[inside], b.m[inside]) and torch.equal(a.v[inside], b.v[inside]), step
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params)), step
