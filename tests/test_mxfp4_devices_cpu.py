"""The calls on MXFP4 weights look at the device of everything that a kernel
reads, the adapter pool and the segments among it (no GPU: the check is watched,
nothing is launched)."""
import pytest
import torch

import segmented_rank_gemm_segment_amd as srg


class Checked(Exception):
    pass


def test_fused_checks_pool_and_segments(monkeypatch):
    def launch_stream(stream, *tensors):
        raise Checked([t for t in tensors if t is not None])
    monkeypatch.setattr(srg, "_launch_stream", launch_stream)
    n, d_in, d_out = 3, 64, 16
    pool = srg.Pool.__new__(srg.Pool)
    pool.A = torch.zeros((2, 8, d_in), dtype=torch.bfloat16)
    pool.Bt = torch.zeros((2, 8, d_out), dtype=torch.bfloat16)
    pool.n_slots, pool.r_max, pool.d_in, pool.d_out, pool.dtype = 2, 8, d_in, d_out, torch.bfloat16
    seg = srg.Segments(n, 2, "cpu")
    X, Y = torch.zeros(n, d_in).bfloat16(), torch.zeros(n, d_out).bfloat16()
    Wq, ws = srg.mxfp4_empty(d_out, d_in, "cpu")
    H = torch.zeros(n, 8)
    with pytest.raises(Checked) as e:
        srg.lora_linear_fused_mxfp4w(X, Wq, ws, H, seg, pool, Y)
    seen = {t.data_ptr() for t in e.value.args[0]}
    for t in (X, Y, Wq, ws, H, pool.A, pool.Bt, seg.row_segment):
        assert t.data_ptr() in seen
