"""Cases for the MXFP4 and expert-routing operators of the multi-LoRA layer.

Five operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and, with ``own`` true, through the calls of
``segmented_rank_gemm_segment_amd``:

* ``quantize``  rows to MXFP4 (E2M1 codes, one E8M0 scale per 32 values) and
                back to the values the codes stand for
* ``linear``    Y = X dq(W)^T (+ s_a (X A_a^T) B_a^T) with an MXFP4 weight and
                bf16 activations, the quantized base of the multi-LoRA layer
* ``product``   Y = dq(q(X)) dq(W)^T: the activations quantized on the way in,
                both operands MXFP4
* ``route``     token choices sorted by expert, rows gathered into that order
                and combined back with the router's weights; with gradients
* ``experts``   the sort and the experts' products on MXFP4 weights, one weight
                per expert

MXFP4 (the OCP microscaling format): 32 consecutive values share the scale
2^(s - 127); a code's value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign;
element 2c of a row is the low half of byte c.  Quantizing a block takes the
scale 2^(floor(log2(amax)) - 2) and rounds to the nearest value, ties to the
even code, past 6 to 6.
"""
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the activations of one decode step on their way to a 4-bit product
        dict(name="quantize_decode", op="quantize", n=256, d=4096, dtype="bf16"),
        # a whole MLP weight at load time
        dict(name="quantize_weight", op="quantize", n=28672, d=8192, dtype="bf16"),
        # one new token through an up projection: the weight's bytes count
        dict(name="linear_token", op="linear", n=1, d_in=8192, d_out=28672, slots=0, r_max=0),
        # a decode batch, every row on its own adapter
        dict(name="linear_decode_lora", op="linear", n=256, d_in=4096, d_out=4096, slots=128,
             r_max=16),
        # a prefill batch of eight requests, each on its adapter, odd number of rows
        dict(name="linear_prefill_lora", op="linear", n=16943, d_in=4096, d_out=14336, slots=8,
             r_max=64),
        # the same product with 4-bit activations on the scaled matrix instructions
        dict(name="product_prefill", op="product", n=16943, d_in=4096, d_out=14336),
        # a chunked prefill's ragged rows on a narrow key/value projection
        dict(name="product_ragged", op="product", n=333, d_in=8192, d_out=1024),
        # routing of a decode batch, latency bound
        dict(name="route_decode", op="route", n=64, top_k=8, experts=128, d=4096, dtype="bf16",
             grad=False, drop=0.0),
        # routing of a training batch, forward and backward
        dict(name="route_train", op="route", n=16384, top_k=4, experts=64, d=4096, dtype="bf16",
             grad=True, drop=0.0),
        # the same in fp32 with odd sizes and padded tokens, whose choices name no expert
        dict(name="route_train_f32", op="route", n=2047, top_k=2, experts=8, d=1032, dtype="f32",
             grad=True, drop=0.1),
        # a decode batch's expert products: few rows on every expert's weight
        dict(name="experts_decode", op="experts", n=64, top_k=8, experts=128, d_in=2048,
             d_out=1536, drop=0.0),
        # a prefill's expert products: long, uneven segments
        dict(name="experts_prefill", op="experts", n=8190, top_k=8, experts=64, d_in=2048,
             d_out=1536, drop=0.02),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _steps(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return min(hi // step, max(lo // step, _log(rng, lo, hi) // step)) * step


def draw(rng):
    op = rng.choice(["quantize", "linear", "product", "route", "experts"])
    if op == "quantize":
        while True:
            c = dict(op=op, n=_log(rng, 1, 28672), d=_steps(rng, 32, 14336, 32),
                     dtype=rng.choice(["bf16", "f32"]))
            if c["n"] * c["d"] <= 28672 * 8192 // 2:
                return c
    if op in ("linear", "product"):
        while True:
            c = dict(op=op, n=_log(rng, 1, 16943), d_in=_steps(rng, 256, 8192, 32),
                     d_out=_steps(rng, 256, 14336, 8))
            if op == "linear":
                c["slots"] = rng.choice([0, _log(rng, 1, 128)])
                c["r_max"] = rng.choice([8, 16, 32, 64]) if c["slots"] else 0
            if c["n"] * c["d_in"] * c["d_out"] <= 16943 * 4096 * 14336:
                return c
    while True:
        experts = _log(rng, 4, 256)
        c = dict(op=op, n=_log(rng, 1, 16384), top_k=rng.randint(1, min(8, experts)),
                 experts=experts, drop=rng.choice([0.0, 0.05, 0.3]))
        if op == "route":
            c.update(d=_steps(rng, 64, 8192, 8), dtype=rng.choice(["bf16", "f32"]),
                     grad=rng.random() < 0.6)
            if c["n"] * c["top_k"] * c["d"] <= 16384 * 4 * 4096 // 2:
                return c
        else:
            c.update(d_in=_steps(rng, 256, 4096, 32), d_out=_steps(rng, 256, 4096, 8))
            if experts * c["d_in"] * c["d_out"] <= 128 * 2048 * 1536 and \
                    c["n"] * c["top_k"] * c["d_in"] * c["d_out"] <= 8190 * 8 * 2048 * 1536:
                return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _activations(g, n, d, dtype):
    """Normal rows with a few large channels and a row scale each, as a
    layer's activations have."""
    x = torch.randn(n, d, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-2, 3, (n, 1), generator=g, device=DEV).float())
    x *= torch.where(torch.rand(1, d, generator=g, device=DEV) < 0.01, 8.0, 1.0)
    return x.to(dtype)


def _mx_weight(g, rows, d):
    """MXFP4 codes [rows, d / 2] and scales [rows, d / 32] of N(0, 0.02)
    weights.  The scale rows are padded to whole 4-byte words."""
    codes = torch.empty(rows, d // 2, dtype=torch.uint8, device=DEV)
    pad = (d // 32 + 3) // 4 * 4
    scales = torch.zeros(rows, pad, dtype=torch.uint8, device=DEV)[:, :d // 32]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = max(1, (1 << 26) // d)
    for r in range(0, rows, step):
        w = torch.randn(min(step, rows - r), d // 32, 32, generator=g, device=DEV) * 0.02
        e = torch.frexp(w.abs().amax(-1)).exponent - 3            # floor(log2(amax)) - 2
        mag = torch.bucketize(torch.ldexp(w.abs(), -e.unsqueeze(-1)), mids)
        code = (mag + 8 * (w < 0)).to(torch.uint8).reshape(w.shape[0], d // 2, 2)
        codes[r:r + step] = code[..., 0] | (code[..., 1] << 4)
        scales[r:r + step] = (e + 127).to(torch.uint8)
    return codes, scales


def _mx_buffers(n, d):
    """Room for the codes and scales of n rows."""
    pad = (d // 32 + 3) // 4 * 4
    return (torch.empty(n, d // 2, dtype=torch.uint8, device=DEV),
            torch.empty(n, pad, dtype=torch.uint8, device=DEV)[:, :d // 32])


def _choices(g, c):
    """The router's choices: top_k distinct experts a token, some experts more
    popular than others; padded tokens name none (-1).  Weights add up to 1."""
    n, k, e = c["n"], c["top_k"], c["experts"]
    liking = torch.randn(1, e, generator=g, device=DEV)
    noise = -torch.log(-torch.log(torch.rand(n, e, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    top = (liking + noise).topk(k, dim=1)
    ids = top.indices.to(torch.int32)
    if c["drop"]:
        ids[torch.rand(n, generator=g, device=DEV) < c["drop"]] = -1
    return ids.contiguous(), torch.softmax(top.values, dim=1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        dt = DTYPES[case["dtype"]]
        s["X"] = _activations(g, case["n"], case["d"], dt)
        s["Xq"], s["xs"] = _mx_buffers(case["n"], case["d"])
        s["out"] = torch.empty(case["n"], case["d"], dtype=dt, device=DEV)
    elif op in ("linear", "product"):
        n, d_in, d_out = case["n"], case["d_in"], case["d_out"]
        s["X"] = _activations(g, n, d_in, torch.bfloat16)
        s["Wq"], s["ws"] = _mx_weight(g, d_out, d_in)
        s["Y"] = torch.empty(n, d_out, dtype=torch.bfloat16, device=DEV)
        if op == "product":
            s["Xq"], s["xs"] = _mx_buffers(n, d_in)
        elif case["slots"]:
            S, r = case["slots"], case["r_max"]
            pick = torch.randint(-1, S, (n,), generator=g, device=DEV, dtype=torch.int32)
            # a batch longer than the slots is requests of many rows each, otherwise decode rows
            s["slot"] = pick if n <= 4 * S else torch.sort(pick).values
            s["rank"] = torch.randint(1, r // 8 + 1, (S,), generator=g, device=DEV,
                                      dtype=torch.int32) * 8
            s["A"] = (torch.randn(S, r, d_in, generator=g, device=DEV) * 0.02).bfloat16()
            s["Bt"] = (torch.randn(S, r, d_out, generator=g, device=DEV) * 0.02).bfloat16()
            s["H"] = torch.empty(n, r, device=DEV)
    else:
        s["ids"], s["w"] = _choices(g, case)
        n, k = case["n"], case["top_k"]
        if op == "route":
            d, dt = case["d"], DTYPES[case["dtype"]]
            s["X"] = _activations(g, n, d, dt)
            s["Ys"] = torch.randn(n * k, d, generator=g, device=DEV).to(dt)
            # rows behind the last routed one are never written
            s["Xs"] = torch.zeros(n * k, d, dtype=dt, device=DEV)
            s["Y"] = torch.empty(n, d, dtype=dt, device=DEV)
            if case["grad"]:
                s["dY"] = torch.randn(n, d, generator=g, device=DEV).to(dt)
                s["dXs"] = torch.randn(n * k, d, generator=g, device=DEV).to(dt)
                s["dYs"] = torch.zeros(n * k, d, dtype=dt, device=DEV)
                s["dw"] = torch.empty(n, k, device=DEV)
                s["dX"] = torch.empty(n, d, dtype=dt, device=DEV)
        else:
            E, d_in, d_out = case["experts"], case["d_in"], case["d_out"]
            s["X"] = _activations(g, n, d_in, torch.bfloat16)
            wq, ws = _mx_weight(g, E * d_out, d_in)
            s["Wq"] = wq.view(E, d_out, d_in // 2)
            s["ws"] = ws.as_strided((E, d_out, d_in // 32), (d_out * ws.stride(0), ws.stride(0), 1))
            s["Y"] = torch.zeros(n * k, d_out, dtype=torch.bfloat16, device=DEV)
            # rows of the fullest expert: the padding of the plain form's batched product
            flat = s["ids"].reshape(-1).long()
            s["most"] = max(1, int(torch.bincount(flat + 1, minlength=E + 1)[1:].max()))
    if own:
        # the handles a program keeps beside its buffers
        import segmented_rank_gemm_segment_amd as srg
        if "A" in s:
            s["pool"] = srg.Pool(s["A"], s["Bt"], s["rank"], 16.0)
            s["seg"] = srg.Segments(case["n"], case["slots"], DEV)
        if "ids" in s:
            s["ex"] = srg.Experts(case["n"], case["top_k"], case["experts"], DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _power(byte):
    """2^(byte - 127) of E8M0 scale bytes, from the bits of a float."""
    b = byte.to(torch.int32)
    return torch.where(b == 0, 2.0 ** -127, (b << 23).view(torch.float32))


def _round_mx(x):
    """The values of x's MXFP4 codes, in float32."""
    b = x.float().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True).view(torch.int32) >> 23       # biased exponent
    byte = (top - 2).clamp(min=0)
    q = b * ((254 - byte) << 23).view(torch.float32)
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.copysign(v, q) * _power(byte)).reshape(x.shape)


def _values(codes, scales):
    """The values of MXFP4 codes and scales, in float32."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    both = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=-1)
    v = both.reshape(*scales.shape, 32) * _power(scales).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], -1)


def _lora(s):
    """s_a (X A_a^T) B_a^T of every row, as two products over all slots' ranks
    with the other slots' entries zeroed."""
    S, r = s["slots"], s["r_max"]
    X = s["X"].float()
    live = torch.arange(r, device=X.device) < s["rank"].unsqueeze(1)              # [S, r]
    scale = torch.where(live, 16.0 / s["rank"].unsqueeze(1).float(), 0.0)
    mine = s["slot"].unsqueeze(1) == torch.arange(S, device=X.device)             # [n, S]
    H = (X @ s["A"].float().reshape(S * r, -1).t()).reshape(-1, S, r)
    H = torch.where(mine.unsqueeze(-1), H * scale, 0.0)
    return H.reshape(-1, S * r) @ s["Bt"].float().reshape(S * r, -1)


def _sort(s):
    """Choices by expert, in order within one: sorted -> choice, choice ->
    sorted (-1 for a dropped one) and each expert's first row."""
    flat = s["ids"].reshape(-1).long()
    E = s["experts"]
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    back = torch.empty_like(order)
    back[order] = torch.arange(order.numel(), device=order.device)
    off = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device=order.device))
    return order, torch.where(key < E, back, -1), off, key


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _round_mx(s["X"]).to(s["X"].dtype)
    if op == "linear":
        Y = s["X"].float() @ _values(s["Wq"], s["ws"]).t()
        return (Y + _lora(s) if s["slots"] else Y).bfloat16()
    if op == "product":
        return (_round_mx(s["X"]) @ _values(s["Wq"], s["ws"]).t()).bfloat16()
    order, back, off, key = _sort(s)
    n, k = s["n"], s["top_k"]
    routed = (key[order] < s["experts"]).unsqueeze(1)
    if op == "route":
        dt = s["X"].dtype
        kept = (back >= 0).unsqueeze(1)
        at = back.clamp(min=0)
        Xs = torch.where(routed, s["X"][order // k], 0)
        ys = torch.where(kept, s["Ys"][at].float(), 0.0).reshape(n, k, -1)
        out = {"position": back.int().reshape(n, k), "offsets": off.int(), "Xs": Xs,
               "Y": (ys * s["w"].unsqueeze(-1)).sum(1).to(dt)}
        if s["grad"]:
            dY = s["dY"].float()
            out["dw"] = (ys * dY.unsqueeze(1)).sum(-1)
            dYs = s["w"].reshape(-1)[order].unsqueeze(1) * dY[order // k]
            out["dYs"] = torch.where(routed, dYs, 0.0).to(dt)
            out["dX"] = torch.where(kept, s["dXs"][at].float(), 0.0).reshape(n, k, -1).sum(1).to(dt)
        return out
    E = s["experts"]
    e = key[order].clamp(max=E - 1)
    place = torch.where(routed.squeeze(1),
                        e * s["most"] + torch.arange(n * k, device=e.device) - off[e], E * s["most"])
    rows = torch.zeros(E * s["most"] + 1, s["d_in"], device=e.device)
    rows[place] = s["X"][order // k].float()
    rows = rows[:-1].reshape(E, s["most"], -1)
    W = _values(s["Wq"], s["ws"]).transpose(1, 2).contiguous()
    Y = torch.bmm(rows, W).reshape(E * s["most"], -1)
    Y = torch.where(routed, Y[place.clamp(max=E * s["most"] - 1)], 0.0)
    return {"offsets": off.int(), "Y": Y.bfloat16()}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import segmented_rank_gemm_segment_amd as srg
    op = s["op"]
    if op == "quantize":
        srg.lora_mxfp4_quantize(s["X"], s["Xq"], s["xs"])
        srg.lora_mxfp4_dequantize(s["Xq"], s["xs"], s["out"])
        return s["out"]
    if op == "linear":
        if not s["slots"]:
            srg.lora_base_gemm_mxfp4w(s["X"], s["Wq"], s["ws"], s["Y"])
        else:
            srg.lora_build_shrink(s["slot"], s["X"], s["pool"], s["seg"], s["H"])
            srg.lora_linear_fused_mxfp4w(s["X"], s["Wq"], s["ws"], s["H"], s["seg"], s["pool"],
                                         s["Y"])
        return s["Y"]
    if op == "product":
        srg.lora_mxfp4_quantize(s["X"], s["Xq"], s["xs"])
        srg.lora_base_gemm_mxfp4(s["Xq"], s["xs"], s["Wq"], s["ws"], s["Y"])
        return s["Y"]
    ex = s["ex"]
    srg.lora_experts_sort(s["ids"], ex)
    if op == "experts":
        srg.lora_experts_gemm_mxfp4w(s["X"], ex, s["Wq"], s["ws"], s["Y"])
        return {"offsets": ex.expert_offsets, "Y": s["Y"]}
    srg.lora_experts_gather(s["X"], ex, s["Xs"])
    srg.lora_experts_combine(s["Ys"], s["w"], ex, s["Y"])
    out = {"position": ex.choice_position, "offsets": ex.expert_offsets, "Xs": s["Xs"],
           "Y": s["Y"]}
    if s["grad"]:
        srg.lora_experts_combine_backward(s["dY"], s["Ys"], s["w"], ex, s["dYs"], s["dw"])
        # the gather's gradient is a combine whose weights are all one
        srg.lora_experts_combine(s["dXs"], None, ex, s["dX"])
        out.update(dw=s["dw"], dYs=s["dYs"], dX=s["dX"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize":
        e = 2 if case["dtype"] == "bf16" else 4
        size = case["n"] * case["d"]
        return {"bytes": size * (2 * e + 17 / 32), "flops": 0}
    if op in ("linear", "product"):
        n, d_in, d_out = case["n"], case["d_in"], case["d_out"]
        size = 2 * n * (d_in + d_out) + d_in * d_out * 17 / 32
        flops = 2 * n * d_in * d_out
        if op == "product":
            size += n * d_in * 17 / 32
        elif case["slots"]:
            r = case["r_max"] / 2 + 4                     # ranks are multiples of 8 up to r_max
            used = case["slots"] * (1 - (1 - 1 / (case["slots"] + 1)) ** n)
            size += 2 * used * r * (d_in + d_out) + 4 * n
            flops += 2 * n * r * (d_in + d_out)
        return {"bytes": size, "flops": flops}
    n, k = case["n"], case["top_k"]
    kept = n * k * (1 - case["drop"])
    if op == "route":
        e = 2 if case["dtype"] == "bf16" else 4
        row = case["d"] * e
        size = n * k * 12 + row * (n + kept) + row * (kept + n)
        flops = 2 * kept * case["d"]
        if case["grad"]:
            size += row * (n + 2 * kept) + n * k * 8 + row * (kept + n)
            flops += 4 * kept * case["d"]
        return {"bytes": size, "flops": flops}
    d_in, d_out, E = case["d_in"], case["d_out"], case["experts"]
    used = E * (1 - (1 - 1 / E) ** kept)
    return {"bytes": n * k * 8 + 2 * n * d_in + 2 * kept * d_out + used * d_in * d_out * 17 / 32,
            "flops": 2 * kept * d_in * d_out}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_power(e):
    """2^e from the bits of a double (pow() may be off in the last place, which
    moves values that lie on a rounding border)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round(x):
    x = x.double()
    out = torch.empty_like(x)
    for r in range(0, x.shape[0], 4096):
        b = x[r:r + 4096].reshape(-1, 32)
        top = b.abs().amax(1)
        e = torch.where(top > 0, torch.frexp(top).exponent - 1, -1000).clamp(min=-125) - 2
        scale = _exact_power(e).unsqueeze(1)
        m = (b / scale).abs()
        code = torch.zeros_like(m)
        for mid, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                            (3.5, True), (5.0, False)):
            code += (m >= mid) if tie_up else (m > mid)
        v = torch.where(code <= 4, code / 2, torch.where(code == 7, 6.0, code - 2))
        out[r:r + 4096] = (torch.sign(b) * v * scale).reshape(-1, x.shape[1])
    return out


def _exact_weight(codes, scales):
    c = torch.stack([codes & 7, codes >> 4 & 7], dim=-1).flatten(-2).double()
    neg = torch.stack([codes & 8, codes >> 4 & 8], dim=-1).flatten(-2) != 0
    v = torch.where(c <= 4, c / 2, torch.where(c == 7, 6.0, c - 2))
    scale = _exact_power(scales.long() - 127)
    return torch.where(neg, -v, v) * scale.repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_round(s["X"])
    if op in ("linear", "product"):
        X = _exact_round(s["X"]) if op == "product" else s["X"].double()
        Y = X @ _exact_weight(s["Wq"], s["ws"]).t()
        if op == "linear" and case["slots"]:
            rank = s["rank"].tolist()
            for a in range(case["slots"]):
                rows = (s["slot"] == a).nonzero().squeeze(1)
                h = X[rows] @ s["A"][a, :rank[a]].double().t()
                Y[rows] += 16.0 / rank[a] * (h @ s["Bt"][a, :rank[a]].double())
        return Y
    n, k, E = case["n"], case["top_k"], case["experts"]
    ids = s["ids"].reshape(-1)
    by_expert = [(ids == e).nonzero().squeeze(1) for e in range(E)]
    order = torch.cat(by_expert)
    if op == "experts":
        Y = torch.zeros(n * k, case["d_out"], dtype=torch.float64, device=DEV)
        at = 0
        for e, rows in enumerate(by_expert):
            Y[at:at + rows.numel()] = s["X"][rows // k].double() @ \
                _exact_weight(s["Wq"][e], s["ws"][e]).t()
            at += rows.numel()
        return {"offsets": None, "Y": Y}
    full = torch.zeros(n * k, case["d"], dtype=torch.float64, device=DEV)

    def to_choices(t):
        full.zero_()
        full[order] = t[:order.numel()].double()
        return full.reshape(n, k, -1)

    Xs = torch.zeros_like(s["Xs"], dtype=torch.float64)
    Xs[:order.numel()] = s["X"].double()[order // k]
    w = s["w"].double()
    out = {"position": None, "offsets": None, "Xs": Xs,
           "Y": torch.matmul(w.unsqueeze(1), to_choices(s["Ys"])).squeeze(1)}
    if case["grad"]:
        dY = s["dY"].double()
        out["dw"] = torch.matmul(to_choices(s["Ys"]), dY.unsqueeze(2)).squeeze(2)
        dYs = torch.zeros_like(Xs)
        dYs[:order.numel()] = (w.unsqueeze(2) * dY.unsqueeze(1)).reshape(n * k, -1)[order]
        out["dYs"] = dYs
        ones = torch.ones_like(w).unsqueeze(1)
        out["dX"] = torch.matmul(ones, to_choices(s["dXs"])).squeeze(1)
    return out
