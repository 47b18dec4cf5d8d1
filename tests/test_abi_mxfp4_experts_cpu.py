"""Refusals of the MXFP4 and expert-routing calls, on the host before any launch
(no GPU: the pointers are fake and never dereferenced)."""
import ctypes
import os

import pytest
import torch

import segmented_rank_gemm_segment_amd as srg

OK, ENULL, ESHAPE, EALIGN, EDTYPE = 0, -1, -2, -4, -5
P = 0x10000


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


def test_quantize_and_dequantize(L):
    q = dict(X=P, ldx=64, n=0, d=64, dtype=1, Xq=P, ldq=32, s=P, lds=4, st=None)
    cases = [({}, OK), (dict(n=-1), ESHAPE), (dict(d=0), ESHAPE), (dict(d=-32), ESHAPE),
             (dict(d=48), EALIGN), (dict(d=40), EALIGN), (dict(dtype=2), EDTYPE),
             (dict(n=1, X=None), ENULL), (dict(n=1, Xq=None), ENULL), (dict(n=1, s=None), ENULL),
             (dict(n=1, ldx=56), ESHAPE), (dict(n=1, ldx=68), EALIGN), (dict(n=1, X=P + 8), EALIGN),
             (dict(n=1, ldq=16), ESHAPE), (dict(n=1, ldq=40), EALIGN), (dict(n=1, Xq=P + 4), EALIGN),
             (dict(n=1, lds=1), ESHAPE), (dict(n=1, lds=6), EALIGN), (dict(n=1, s=P + 4), EALIGN),
             (dict(n=1, ldx=(1 << 22) + 8), ESHAPE), (dict(n=1, ldq=(1 << 22) + 16), ESHAPE),
             (dict(n=1, d=(1 << 22) + 32), ESHAPE)]
    vary(L.lora_mxfp4_quantize, q, cases)
    order = ("Xq", "ldq", "s", "lds", "n", "d", "dtype", "X", "ldx", "st")
    vary(L.lora_mxfp4_dequantize, {k: q[k] for k in order}, cases)


def test_products(L):
    a = dict(X=P, ldx=64, Wq=P, ldw=32, ws=P, ldws=4, Y=P, ldy=16, n=0, d_in=64, d_out=16, st=None)
    vary(L.lora_base_gemm_mxfp4w, a, [
        ({}, OK), (dict(n=-1), ESHAPE), (dict(d_in=0), ESHAPE), (dict(d_out=0), ESHAPE),
        (dict(d_in=48), EALIGN), (dict(d_out=12), EALIGN), (dict(Wq=None), ENULL),
        (dict(ws=None), ENULL), (dict(ldw=16), ESHAPE), (dict(ldw=40), EALIGN),
        (dict(ldws=1), ESHAPE), (dict(ldws=7), EALIGN), (dict(Wq=P + 8), EALIGN),
        (dict(ws=P + 8), EALIGN), (dict(n=1, X=None), ENULL), (dict(n=1, Y=None), ENULL),
        (dict(n=1, ldx=56), ESHAPE), (dict(n=1, ldx=68), EALIGN), (dict(n=1, ldy=8), ESHAPE),
        (dict(n=1, Y=P + 2), EALIGN)])
    b = dict(Xq=P, ldx=32, xs=P, ldxs=4, Wq=P, ldw=32, ws=P, ldws=4, Y=P, ldy=16, n=0, d_in=64,
             d_out=16, st=None)
    vary(L.lora_base_gemm_mxfp4, b, [
        ({}, OK), (dict(n=-1), ESHAPE), (dict(d_in=96, n=1), ESHAPE), (dict(d_in=72), EALIGN),
        (dict(n=1, Xq=None), ENULL), (dict(n=1, xs=None), ENULL), (dict(n=1, ldx=16), ESHAPE),
        (dict(n=1, ldx=36), EALIGN), (dict(n=1, ldxs=5), EALIGN), (dict(n=1, Y=None), ENULL),
        (dict(Wq=None), ENULL), (dict(ldws=0), ESHAPE)])


def test_fused(L):
    def pool(**kw):
        d = dict(n_slots=4, r_max=16, d_in=64, d_out=32, dtype=1, rank_policy=0, A=P, Bt=P,
                 slot_rank=P, slot_scale=P)
        d.update(kw)
        return srg.LoraPoolC(**d)
    seg = srg.LoraSegmentsC(n_rows=10, max_segments=5, token_indices=P, row_segment=P,
                            segment_offsets=P, segment_slots=P, segment_ranks=P, segment_scales=P,
                            num_segments=P, status=P)

    def call(p=None, seg_=seg, X=P, ldx=64, Wq=P, ldw=32, ws=P, ldws=4, H=P, Y=P, ldy=32):
        p = pool() if p is None else p
        return L.lora_linear_fused_mxfp4w(X, ldx, Wq, ldw, ws, ldws, H, seg_ and ctypes.byref(seg_),
                                          ctypes.byref(p), Y, ldy, None)
    assert L.lora_linear_fused_mxfp4w(P, 64, P, 32, P, 4, P, ctypes.byref(seg), None, P, 32, None) == ENULL
    assert call(pool(dtype=0)) == EDTYPE
    assert call(pool(d_in=40)) == EALIGN
    assert call(seg_=None) == ENULL
    assert call(Wq=None) == ENULL and call(ws=None) == ENULL and call(H=None) == ENULL
    assert call(X=None) == ENULL and call(Y=None) == ENULL
    assert call(ldw=16) == ESHAPE and call(ldws=6) == EALIGN and call(H=P + 4) == EALIGN
    assert call(ldy=24) == ESHAPE


def experts(**kw):
    d = dict(n_tokens=10, top_k=2, n_experts=4, expert_offsets=P, sorted_choice=P,
             choice_position=P, status=P, workspace=P)
    d.update(kw)
    return srg.LoraExpertsC(**d)


BAD_EXPERTS = [
    (dict(n_tokens=-1), ESHAPE), (dict(top_k=0), ESHAPE), (dict(top_k=65), ESHAPE),
    (dict(n_experts=0), ESHAPE), (dict(n_experts=1025), ESHAPE),
    (dict(n_tokens=(1 << 29) + 1), ESHAPE), (dict(expert_offsets=None), ENULL),
    (dict(status=None), ENULL), (dict(sorted_choice=None), ENULL), (dict(choice_position=None), ENULL),
]


def test_sort(L):
    for change, want in BAD_EXPERTS:
        assert L.lora_experts_sort(P, ctypes.byref(experts(**change)), None) == want, change
    assert L.lora_experts_sort(P, None, None) == ENULL
    assert L.lora_experts_sort(None, ctypes.byref(experts()), None) == ENULL
    big = experts(n_tokens=100000, workspace=None)
    assert L.lora_experts_sort(P, ctypes.byref(big), None) == ENULL
    assert L.lora_experts_workspace(64, 8, 128) == 0
    assert L.lora_experts_workspace(0, 1, 1) == 0
    assert L.lora_experts_workspace(100000, 8, 128) > 0
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 2, 1)):
        assert L.lora_experts_workspace(*bad) == -1


def test_rows(L):
    ex, none = ctypes.byref(experts()), ctypes.byref(experts(n_tokens=0))
    g = dict(X=P, ldx=64, ex=ex, d=64, dtype=1, Xs=P, lds=64, st=None)
    cases = [(dict(ex=None), ENULL), (dict(d=0), ESHAPE), (dict(d=12), EALIGN), (dict(dtype=3), EDTYPE),
             (dict(X=None), ENULL), (dict(ldx=56), ESHAPE), (dict(ldx=66), EALIGN), (dict(Xs=None), ENULL),
             (dict(lds=32), ESHAPE), (dict(Xs=P + 8), EALIGN), (dict(ex=none), OK)]
    cases += [(dict(ex=ctypes.byref(experts(**c))), w) for c, w in BAD_EXPERTS]
    vary(L.lora_experts_gather, g, cases)
    c = dict(X=P, ldx=64, w=None, ex=ex, d=64, dtype=0, Xs=P, lds=64, st=None)
    vary(L.lora_experts_combine, c, cases)
    b = dict(dY=P, lddy=64, Ys=P, ldys=64, w=None, ex=ex, d=64, dtype=1, dYs=P, lddys=64, dw=P, st=None)
    vary(L.lora_experts_combine_backward, b, [
        (dict(ex=None), ENULL), (dict(dY=None), ENULL), (dict(Ys=None), ENULL),
        (dict(dYs=None, dw=None), ENULL), (dict(lddys=56), ESHAPE), (dict(ldys=60), ESHAPE),
        (dict(dYs=P + 8), EALIGN), (dict(d=4), EALIGN), (dict(dtype=-1), EDTYPE), (dict(ex=none), OK)])


def test_experts_product(L):
    a = dict(X=P, ldx=64, g=1, ex=ctypes.byref(experts()), Wq=P, ldw=32, ws=P, ldws=4, Y=P, ldy=16,
             d_in=64, d_out=16, st=None)
    cases = [(dict(ex=None), ENULL), (dict(d_in=40), EALIGN), (dict(d_out=4), EALIGN), (dict(d_in=0), ESHAPE),
             (dict(Wq=None), ENULL), (dict(ws=None), ENULL), (dict(ldw=16), ESHAPE), (dict(ldws=2), EALIGN),
             (dict(X=None), ENULL), (dict(Y=None), ENULL), (dict(ldx=32), ESHAPE), (dict(ldy=20), EALIGN),
             (dict(ex=ctypes.byref(experts(n_tokens=0))), OK)]
    cases += [(dict(ex=ctypes.byref(experts(**c))), w) for c, w in BAD_EXPERTS]
    vary(L.lora_experts_gemm_mxfp4w, a, cases)


def test_tensor_checks():
    """The binding's own refusals, before any pointer is passed on."""
    q, s = srg.mxfp4_empty(4, 64, "cpu")
    assert q.shape == (4, 32) and s.shape == (4, 2) and s.stride(0) == 4
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        srg.mxfp4_empty(4, 40, "cpu")
    with pytest.raises(ValueError):
        srg.lora_mxfp4_quantize(x, q[:, :16], s)
    with pytest.raises(ValueError):
        srg.lora_mxfp4_quantize(x, q.to(torch.int32), s)
    with pytest.raises(ValueError):
        srg.lora_base_gemm_mxfp4w(x, q, s, torch.zeros(4, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        srg.lora_base_gemm_mxfp4w(x.bfloat16(), q, s, torch.zeros(4, 8, dtype=torch.bfloat16))
    for bad in ((4, 0, 2), (4, 65, 2), (4, 1, 0), (4, 1, 1025), (-1, 1, 1)):
        with pytest.raises(ValueError):
            srg.Experts(*bad, device="cpu")
    ex = srg.Experts(4, 2, 3, "cpu")
    with pytest.raises(ValueError):
        srg.lora_experts_sort(torch.zeros(4, 2, dtype=torch.int64), ex)
    with pytest.raises(ValueError):
        srg.lora_experts_sort(torch.zeros(4, 3, dtype=torch.int32), ex)
    with pytest.raises(ValueError):
        srg.lora_experts_gather(x, ex, torch.zeros(4, 64))
    with pytest.raises(ValueError):
        srg.lora_experts_combine(torch.zeros(8, 64), torch.zeros(4, 2, dtype=torch.float64), ex, x)
    with pytest.raises(ValueError):
        srg.lora_experts_combine(torch.zeros(8, 64).bfloat16(), None, ex, x)
    w3 = torch.zeros(3, 16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        srg.lora_experts_gemm_mxfp4w(x.bfloat16(), ex, w3[:2], torch.zeros(3, 16, 4, dtype=torch.uint8)[:2, :, :2],
                                     torch.zeros(8, 16, dtype=torch.bfloat16))


def test_rows_past_the_limit(L):
    big = (1 << 28) + 1
    assert L.lora_mxfp4_quantize(P, 64, big, 64, 1, P, 32, P, 4, None) == ESHAPE
    assert L.lora_mxfp4_dequantize(P, 32, P, 4, big, 64, 1, P, 64, None) == ESHAPE
    assert L.lora_base_gemm_mxfp4w(P, 64, P, 32, P, 4, P, 16, big, 64, 16, None) == ESHAPE
    assert L.lora_base_gemm_mxfp4(P, 32, P, 4, P, 32, P, 4, P, 16, big, 64, 16, None) == ESHAPE
    ex = srg.LoraExpertsC(big, 1, 4, P, P, P, P, P)
    assert L.lora_experts_gemm_mxfp4w(P, 64, 1, ctypes.byref(ex), P, 32, P, 4, P, 16, 64, 16,
                                      None) == ESHAPE


def test_stream_of_another_device(monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    X = torch.zeros(1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        srg.lora_mxfp4_quantize(X, *srg.mxfp4_empty(1, 64, "cpu"), stream=Stream())
