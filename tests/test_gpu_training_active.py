"""The optimizer's `active` formed on the device from a batch's slots, as the README has it:
no host synchronization, and part of a captured step."""
import pytest
import torch

from test_gpu_training_step import DEV, Step

pytestmark = pytest.mark.gpu


def slots_with_rows(slot, live):
    """Into live int32 [n_slots + 1], whose last entry stands for rows without an adapter:
    1 for every slot that a row names."""
    S = live.numel() - 1
    live.zero_().index_fill_(0, torch.where((slot >= 0) & (slot < S), slot, S).long(), 1)
    return live[:S]


def test_rows_that_name_no_slot():
    live = torch.full((6,), 9, dtype=torch.int32, device=DEV)
    slot = torch.tensor([3, -1, 0, 3, 5, 1000, -7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    assert slots_with_rows(slot, live).tolist() == [1, 0, 0, 1, 0]
    assert slots_with_rows(slot[:0], live).tolist() == [0] * 5


def test_captured_step():
    """A captured step whose `active` follows the batch: idle slots keep their weights, moments
    and step counts although their old gradients are still there."""
    c, e = Step(6), Step(6)
    live = torch.zeros(c.S + 1, dtype=torch.int32, device=DEV)

    def run(s, on_device):
        s.forward()
        s.backward()
        if on_device:
            s.active.copy_(slots_with_rows(s.slot, live).repeat(2))
        s.update(seed=3)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(c, True)
    for i in range(4):
        c.batch(idle=i % c.S)
        e.batch(idle=i % e.S)
        c.active.fill_(1)                                # what the graph has to replace
        kept = [t.clone() for t in (c.pool.A[i % c.S], c.pool.Bt[i % c.S])]
        torch.cuda.synchronize()
        graph.replay()
        run(e, False)
        torch.cuda.synchronize()
        assert torch.equal(c.active, e.active)
        assert all(torch.equal(x, y) for x, y in zip(c.everything(), e.everything()))
        assert torch.equal(kept[0], c.pool.A[i % c.S]) and torch.equal(kept[1], c.pool.Bt[i % c.S])
    assert (c.adapters.step < 4).any()
