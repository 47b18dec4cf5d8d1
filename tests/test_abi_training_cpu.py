"""Refusals of the training calls, on the host before any launch (no GPU: the pointers
are fake and never dereferenced, but for the optimizer's table, which is host memory)."""
import ctypes
import os

import pytest
import torch

import segmented_rank_gemm_segment_amd as srg

OK, ENULL, ESHAPE, ERANK, EALIGN, EDTYPE, ECAP = 0, -1, -2, -3, -4, -5, -6
P = 0x10000
BF16 = torch.bfloat16


@pytest.fixture(scope="session")
def L():
    if not os.path.exists(srg.LIB_PATH):
        from segmented_rank_gemm_segment_amd import build
        build.build()
    return srg.lib()


def vary(call, args, cases):
    for change, want in cases:
        a = dict(args)
        a.update(change)
        assert call(*a.values()) == want, (change, want)


# --------------------------------------------------------------- adapters' gradients
def pool(**kw):
    d = dict(n_slots=4, r_max=16, d_in=64, d_out=32, dtype=1, rank_policy=0, A=P, Bt=P,
             slot_rank=P, slot_scale=P)
    d.update(kw)
    return ctypes.byref(srg.LoraPoolC(**d))


def segs(**kw):
    d = dict(n_rows=10, max_segments=5, token_indices=P, row_segment=P, segment_offsets=P,
             segment_slots=P, segment_ranks=P, segment_scales=P, num_segments=P, status=P)
    d.update(kw)
    return ctypes.byref(srg.LoraSegmentsC(**d))


def test_linear_backward(L):
    a = dict(dY=P, lddy=32, Wt=P, ldwt=32, X=P, ldx=64, H=P, seg=segs(), pool=pool(), dH=P, dX=P,
             lddx=64, dA=P, dBt=P, acc=0, st=None)
    cols = (ctypes.c_int32 * 3)(0, 16, 32)
    stacked = pool(r_max=32, n_proj=2, proj_cols=ctypes.cast(cols, ctypes.c_void_p).value)
    vary(L.lora_linear_backward, a, [
        (dict(pool=None), ENULL), (dict(seg=None), ENULL), (dict(pool=pool(dtype=2)), EDTYPE),
        (dict(pool=pool(r_max=12)), ERANK), (dict(pool=pool(d_in=60)), EALIGN),
        (dict(pool=pool(dora_scale=P)), ESHAPE), (dict(pool=stacked), ESHAPE),
        (dict(seg=segs(n_rows=-1)), ESHAPE), (dict(seg=segs(max_segments=4)), ECAP),
        (dict(seg=segs(row_segment=None)), ENULL),
        (dict(dY=None), ENULL), (dict(lddy=24), ESHAPE), (dict(lddy=36), EALIGN),
        (dict(dY=P + 2), EALIGN), (dict(lddy=(1 << 22) + 8), ESHAPE),
        (dict(Wt=None), ENULL), (dict(ldwt=24), ESHAPE), (dict(Wt=P + 8), EALIGN),
        (dict(dX=P + 8), EALIGN), (dict(lddx=56), ESHAPE), (dict(lddx=68), EALIGN),
        (dict(X=None), ENULL), (dict(ldx=56), ESHAPE), (dict(X=P + 4), EALIGN),
        (dict(dA=P + 4), EALIGN), (dict(dBt=P + 8), EALIGN), (dict(dH=None), ENULL),
        (dict(dH=P + 4), EALIGN), (dict(H=None), ENULL), (dict(H=P + 8), EALIGN),
        (dict(seg=segs(n_rows=0)), OK),
        (dict(seg=segs(n_rows=0), dY=None, Wt=None, X=None, H=None, dH=None, dX=None), OK)])
    # what a call leaves out is not asked for
    a["seg"] = segs(n_rows=0)
    vary(L.lora_linear_backward, a, [
        (dict(dX=None, Wt=None, ldwt=0, lddx=0), OK), (dict(dA=None, X=None, ldx=0), OK),
        (dict(dBt=None, H=None), OK)])


def test_linear_backward_binding():
    n, S, R, K, N = 5, 3, 8, 32, 16

    class FakePool:          # (a pool's constructor launches)
        n_proj, dora_scale, dtype, r_max, d_in, d_out = 1, None, BF16, R, K, N
        A, Bt = torch.zeros(S, R, K, dtype=BF16), torch.zeros(S, R, N, dtype=BF16)
    seg = srg.Segments(n, S, "cpu")
    f32 = torch.float32
    good = dict(dY=torch.zeros(n, N, dtype=BF16), Wt=torch.zeros(K, N, dtype=BF16),
                X=torch.zeros(n, K, dtype=BF16), H=torch.zeros(n, R), seg=seg, pool=FakePool(),
                dH=torch.zeros(n, R), dX=torch.zeros(n, K, dtype=BF16), dA=torch.zeros(S, R, K),
                dBt=torch.zeros(S, R, N))
    for change in (dict(dY=torch.zeros(n, N)), dict(dY=torch.zeros(n + 1, N, dtype=BF16)),
                   dict(Wt=torch.zeros(N, K, dtype=BF16)), dict(X=torch.zeros(n, K)),
                   dict(dX=torch.zeros(n, N, dtype=BF16)), dict(Wt=None), dict(X=None), dict(H=None),
                   dict(H=torch.zeros(n, R, dtype=BF16)), dict(dH=torch.zeros(R, n, dtype=f32).T),
                   dict(dH=torch.zeros(n, 2 * R)), dict(dA=torch.zeros(S, R, K, dtype=BF16)),
                   dict(dBt=torch.zeros(S, N, R)), dict(dA=torch.zeros(S, K, R).transpose(1, 2))):
        with pytest.raises(ValueError):
            srg.lora_linear_backward(**dict(good, **change))
    for name, value in (("n_proj", 2), ("dora_scale", torch.ones(S, N))):
        bad = FakePool()
        setattr(bad, name, value)
        with pytest.raises(ValueError, match="one projection"):
            srg.lora_linear_backward(**dict(good, pool=bad))


# --------------------------------------------------------------- experts' products
def experts(**kw):
    d = dict(n_tokens=10, top_k=2, n_experts=4, expert_offsets=P, sorted_choice=P,
             choice_position=P, status=P, workspace=P)
    d.update(kw)
    return ctypes.byref(srg.LoraExpertsC(**d))


BAD_EXPERTS = [
    (dict(n_tokens=-1), ESHAPE), (dict(top_k=0), ESHAPE), (dict(top_k=65), ESHAPE),
    (dict(n_experts=0), ESHAPE), (dict(n_experts=1025), ESHAPE),
    (dict(n_tokens=(1 << 29) + 1), ESHAPE), (dict(expert_offsets=None), ENULL),
    (dict(status=None), ENULL), (dict(sorted_choice=None), ENULL), (dict(choice_position=None), ENULL),
]


def test_experts_gemm(L):
    a = dict(X=P, ldx=64, g=1, ex=experts(), W=P, ldw=64, Y=P, ldy=16, d_in=64, d_out=16, st=None)
    cases = [(dict(ex=None), ENULL), (dict(d_in=0), ESHAPE), (dict(d_out=-8), ESHAPE),
             (dict(d_in=60), EALIGN), (dict(d_out=12), EALIGN), (dict(W=None), ENULL),
             (dict(ldw=56), ESHAPE), (dict(ldw=68), EALIGN), (dict(W=P + 8), EALIGN),
             (dict(ldw=(1 << 22) + 8), ESHAPE), (dict(X=None), ENULL), (dict(ldx=32), ESHAPE),
             (dict(ldx=66), EALIGN), (dict(X=P + 2), EALIGN), (dict(Y=None), ENULL),
             (dict(ldy=8), ESHAPE), (dict(ldy=20), EALIGN), (dict(Y=P + 4), EALIGN),
             (dict(ex=experts(n_tokens=0)), OK), (dict(ex=experts(n_tokens=0), X=None, Y=None), OK)]
    cases += [(dict(ex=experts(**c)), w) for c, w in BAD_EXPERTS]
    vary(L.lora_experts_gemm, a, cases)


def test_experts_gemm_backward(L):
    a = dict(dY=P, lddy=16, X=P, ldx=64, g=1, ex=experts(), W=P, ldw=64, dXs=P, lddxs=64, dW=P,
             lddw=64, dt=1, acc=0, d_in=64, d_out=16, st=None)
    cases = [(dict(ex=None), ENULL), (dict(d_in=0), ESHAPE), (dict(d_out=0), ESHAPE),
             (dict(d_in=60), EALIGN), (dict(d_out=12), EALIGN), (dict(dXs=None, dW=None), ENULL),
             (dict(dt=2), EDTYPE), (dict(dt=-1), EDTYPE), (dict(dY=None), ENULL),
             (dict(lddy=8), ESHAPE), (dict(lddy=18), EALIGN), (dict(dY=P + 8), EALIGN),
             (dict(W=None), ENULL), (dict(ldw=56), ESHAPE), (dict(dXs=P + 8), EALIGN),
             (dict(lddxs=56), ESHAPE), (dict(lddxs=66), EALIGN), (dict(dW=P + 8), EALIGN),
             (dict(lddw=56), ESHAPE), (dict(lddw=66), EALIGN), (dict(X=None), ENULL),
             (dict(ldx=32), ESHAPE), (dict(X=P + 8), EALIGN),
             # without tokens there is nothing for dXs
             (dict(ex=experts(n_tokens=0), dW=None), OK),
             (dict(ex=experts(n_tokens=0), dW=None, dY=None, X=None, dXs=P), OK)]
    cases += [(dict(ex=experts(**c)), w) for c, w in BAD_EXPERTS]
    vary(L.lora_experts_gemm_backward, a, cases)


def test_experts_binding():
    ex = srg.Experts(4, 2, 3, "cpu")
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)
    good = dict(X=z(4, 64), ex=ex, W=z(3, 16, 64), Y=z(8, 16))
    for change in (dict(X=z(4, 64, dtype=torch.float32)), dict(X=z(8, 64)), dict(W=z(2, 16, 64)),
                   dict(W=z(3, 64, 16)), dict(W=z(3, 64, 16).transpose(1, 2)),
                   dict(W=z(3, 32, 64)[:, :16]), dict(W=z(1, 16, 64).expand(3, 16, 64)),
                   dict(Y=z(4, 16)), dict(Y=z(8, 16, dtype=torch.float32)), dict(gathered=False)):
        with pytest.raises(ValueError):
            srg.lora_experts_gemm(**dict(good, **change))
    back = dict(dY=z(8, 16), X=z(4, 64), ex=ex, W=z(3, 16, 64), dXs=z(8, 64), dW=z(3, 16, 64))
    for change in (dict(dY=z(8, 16, dtype=torch.float32)), dict(dY=z(4, 16)), dict(X=z(8, 64)),
                   dict(X=None), dict(W=None), dict(W=z(3, 16, 32)), dict(dXs=z(4, 64)),
                   dict(dXs=None, dW=None), dict(dW=z(3, 16, 64, dtype=torch.float64)),
                   dict(dW=z(1, 16, 64).expand(3, 16, 64)), dict(gathered=False)):
        with pytest.raises(ValueError):
            srg.lora_experts_gemm_backward(**dict(back, **change))


# --------------------------------------------------------------- optimizer
def tensors(*ts):
    a = (srg.LoraAdamwTensorC * len(ts))()
    for i, t in enumerate(ts):
        a[i] = srg.LoraAdamwTensorC(*t)
    return a


G = 0x100000000       # gradients far from the tensors
M = 0x200000000       # and the masters


def table(L, ts, p=1, g=1, n=None, off=0):
    a = tensors(*ts)
    n = len(ts) if n is None else n
    size = max(L.lora_adamw_table_bytes(a, n), 64)
    buf = ctypes.create_string_buffer(size + 32)
    at = (ctypes.addressof(buf) + 15) // 16 * 16 + off
    return L.lora_adamw_table(a, n, p, g, at)


def test_adamw_sizes(L):
    a = tensors((P, G, None, 1), (P, G, None, 256), (P, G, None, 0), (P, G, None, 257))
    assert L.lora_adamw_state_numel(a, 4) == 256 + 256 + 0 + 512
    assert L.lora_adamw_table_bytes(a, 4) > L.lora_adamw_table_bytes(a, 3) > 0
    for bad in (tensors((P, G, None, -1)), tensors((P, G, None, (1 << 40) + 1))):
        assert L.lora_adamw_state_numel(bad, 1) == L.lora_adamw_table_bytes(bad, 1) == -1
        assert L.lora_adamw_table(bad, 1, 1, 1, P) == ESHAPE
    for n in (0, -1, (1 << 20) + 1):
        assert L.lora_adamw_state_numel(a, n) == L.lora_adamw_table_bytes(a, n) == -1
        assert L.lora_adamw_table(a, n, 1, 1, P) == ESHAPE
    assert L.lora_adamw_state_numel(None, 1) == L.lora_adamw_table_bytes(None, 1) == -1
    top = tensors((P, G, None, 1 << 40))
    assert L.lora_adamw_state_numel(top, 1) == 1 << 40


def test_adamw_table(L):
    far = lambda i, n=100: (P + 0x10000 * i, G + 0x10000 * i, None, n)
    assert table(L, [far(0), far(1), far(2, 0)]) == OK
    assert table(L, [(None, None, None, 0), far(1)]) == OK
    assert L.lora_adamw_table(None, 1, 1, 1, P) == ENULL
    assert L.lora_adamw_table(tensors(far(0)), 1, 1, 1, None) == ENULL
    assert table(L, [far(0)], off=4) == EALIGN
    assert table(L, [far(0)], p=2) == EDTYPE and table(L, [far(0)], g=-1) == EDTYPE
    assert table(L, [(None, G, None, 1)]) == ENULL and table(L, [(P, None, None, 1)]) == ENULL
    assert table(L, [(P + 2, G, None, 1)]) == EALIGN and table(L, [(P, G + 8, None, 1)]) == EALIGN
    assert table(L, [(P, G, M + 4, 1)]) == EALIGN
    # masters: for all or none, beside bf16 tensors
    assert table(L, [(P, G, M, 100), (P + 256, G + 256, M + 512, 100)]) == OK
    assert table(L, [(P, G, M, 100), far(1)]) == ESHAPE
    assert table(L, [(P, G, M, 100)], p=0) == ESHAPE
    # what is written overlaps nothing: 100 bf16 elements are 200 bytes
    assert table(L, [(P, G, None, 100), (P + 208, G + 208, None, 100)]) == OK
    assert table(L, [(P, G, None, 100), (P + 192, G + 208, None, 100)]) == ESHAPE
    assert table(L, [(P, G, None, 100), (P + 208, P + 400, None, 100)]) == ESHAPE
    assert table(L, [(P, P, None, 100)]) == ESHAPE
    assert table(L, [(P, G, None, 100), (P, G, None, 100)]) == ESHAPE
    assert table(L, [(P, G, M, 100), (P + 256, G + 256, M + 384, 100)]) == ESHAPE
    assert table(L, [(P, G, P + 192, 100)]) == ESHAPE
    # gradients may be one buffer for several tensors (they are read only)
    assert table(L, [(P, G, None, 100), (P + 256, G, None, 100)]) == OK
    # a long tensor that holds a short one, which is not its neighbour in order
    assert table(L, [(P, G, None, 4096), (P + 16, G, None, 1), (P + 4096, G, None, 1)]) == ESHAPE


def opt(L, **kw):
    a = tensors((P, G, None, 300), (P + 0x1000, G + 0x1000, None, 5))
    d = dict(n_tensors=2, param_dtype=1, grad_dtype=1, masters=0, state_bits=8, state_numel=768,
             table=P, table_bytes=L.lora_adamw_table_bytes(a, 2), m=P, v=P, m_scale=P, v_scale=P,
             step=P)
    d.update(kw)
    return ctypes.byref(srg.LoraAdamwC(**d))


BAD_OPT = [(dict(n_tensors=0), ESHAPE), (dict(n_tensors=(1 << 20) + 1), ESHAPE),
           (dict(param_dtype=2), EDTYPE), (dict(grad_dtype=-1), EDTYPE), (dict(state_bits=16), EDTYPE),
           (dict(masters=1, param_dtype=0), ESHAPE), (dict(state_numel=-256), ESHAPE),
           (dict(state_numel=300), ESHAPE), (dict(table_bytes=8), ESHAPE), (dict(table=None), ENULL),
           (dict(step=None), ENULL), (dict(table=P + 8), EALIGN), (dict(step=P + 2), EALIGN),
           (dict(m=None), ENULL), (dict(v=None), ENULL), (dict(m_scale=None), ENULL),
           (dict(v_scale=None), ENULL), (dict(m=P + 8), EALIGN), (dict(v=P + 4), EALIGN),
           (dict(m_scale=P + 4), EALIGN), (dict(v_scale=P + 8), EALIGN)]


def test_adamw_step(L):
    a = dict(opt=opt(L), lr=1e-3, lr_dev=None, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, gs=None,
             active=None, seed=0, st=None)
    nan, inf = float("nan"), float("inf")
    cases = [(dict(opt=None), ENULL), (dict(lr=nan), ESHAPE), (dict(lr=inf), ESHAPE),
             (dict(b1=1.0), ESHAPE), (dict(b1=-0.1), ESHAPE), (dict(b1=nan), ESHAPE),
             (dict(b2=1.0), ESHAPE), (dict(b2=-1e-9), ESHAPE), (dict(b2=nan), ESHAPE),
             (dict(eps=0.0), ESHAPE), (dict(eps=-1e-8), ESHAPE), (dict(eps=nan), ESHAPE),
             (dict(eps=inf), ESHAPE), (dict(eps=1e-39), ESHAPE), (dict(eps=1e39), ESHAPE),
             (dict(wd=-0.1), ESHAPE), (dict(wd=nan), ESHAPE), (dict(wd=inf), ESHAPE),
             (dict(lr_dev=P + 2), EALIGN), (dict(gs=P + 1), EALIGN), (dict(active=P + 2), EALIGN)]
    cases += [(dict(opt=opt(L, **c)), w) for c, w in BAD_OPT]
    vary(L.lora_adamw_step, a, cases)


def test_adamw_read(L):
    a = dict(opt=opt(L), dtype=1, m=P, v=P, st=None)
    cases = [(dict(opt=None), ENULL), (dict(dtype=2), EDTYPE), (dict(m=None), ENULL),
             (dict(v=None), ENULL), (dict(m=P + 8), EALIGN), (dict(v=P + 2), EALIGN),
             (dict(opt=opt(L, state_bits=32, m_scale=None, v_scale=None)), EDTYPE),
             (dict(opt=opt(L, state_numel=0), m=None, v=None), OK)]
    cases += [(dict(opt=opt(L, **c)), w) for c, w in BAD_OPT]
    vary(L.lora_adamw_read, a, cases)


def test_adamw_binding(L):
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)
    f32 = torch.float32
    w = [z(16, 32), z(300)]
    g = [z(16, 32), z(300)]
    for params, grads, kw in (
            ([], [], {}), (w, g[:1], {}), (w, g, dict(bits=16)), (w, [g[0], z(301)], {}),
            (w, [g[0], z(300, dtype=f32)], {}), ([w[0], z(300, dtype=f32)], g, {}),
            ([z(32, 16).T, w[1]], g, {}), (w, [z(32, 16).T, g[1]], {}),
            ([t.float() for t in w], g, dict(masters=True)), (w, g, dict(masters=[w[0].float()])),
            (w, g, dict(masters=[w[0].float(), w[1]])),
            ([t.half() for t in w], g, {}), (w, [t.half() for t in g], {})):
        with pytest.raises(ValueError):
            srg.AdamW(params, grads, **kw)
    for params, grads in (([w[0], w[0]], [g[0], z(16, 32)]), ([w[0]], [w[0]]),
                          ([z(64)[4:36], w[1]], [z(32), g[1]])):
        with pytest.raises(srg.LoraError):
            srg.AdamW(params, grads)
    o = srg.AdamW(w, g, bits=8)
    assert o.numel == 512 + 512 and o.starts == [0, 512] and o.m_scale.numel() == 4
    for kw in (dict(lr=z(1)), dict(lr=z(2, dtype=f32)), dict(lr=1e-3, grad_scale=z(1)),
               dict(lr=1e-3, active=z(2, dtype=torch.int64)), dict(lr=1e-3, active=z(3, dtype=torch.int32)),
               dict(lr=1e-3, active=z(4, dtype=torch.int32)[::2])):
        with pytest.raises(ValueError):
            srg.lora_adamw_step(o, **kw)
    for m, v in ((z(1000), z(1000)), (z(1024), z(1024, dtype=f32)), (z(2048)[::2], z(1024)),
                 (z(1024).half(), z(1024).half())):
        with pytest.raises(ValueError):
            srg.lora_adamw_read(o, m, v)


def test_stream_of_another_device(monkeypatch, L):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    o = srg.AdamW([torch.zeros(8)], [torch.zeros(8)])
    ex = srg.Experts(4, 2, 3, "cpu")
    z = lambda *s: torch.zeros(*s, dtype=BF16)
    with pytest.raises(ValueError, match="current device"):
        srg.lora_adamw_step(o, 1e-3, stream=Stream())
    with pytest.raises(ValueError, match="current device"):
        srg.lora_experts_gemm(z(4, 64), ex, z(3, 16, 64), z(8, 16), stream=Stream())
    with pytest.raises(ValueError, match="current device"):
        srg.lora_experts_gemm_backward(z(8, 16), None, ex, z(3, 16, 64), z(8, 64), None,
                                       stream=Stream())
