"""AdamW at the ends of its ranges: codes next to the border between two of them.

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
