"""Buffers with the int8 payload on the GPU."""

import pytest

from combine_moe_layout_02_gb300 import inputs, moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first_use", ["dispatch", "property"])
def test_the_4_bit_rows_of_both_payloads_are_the_same(first_use):
    """expert_plan, fp4_rows and dispatch_expert_fp4 with quant = 1 as with 0, on a stream that is not the current one."""
    import torch

    w = inputs.make(2, 8, 100, 256, 3, seed=1, expert_alignment=128)
    x = torch.from_numpy(w.x_bits.view("int16")).cuda().view(torch.bfloat16)
    idx, weights = torch.from_numpy(w.topk_idx).cuda(), torch.from_numpy(w.topk_weights).cuda()
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    for quant in (0, 1):
        buf = moe.Buffers(moe.make_shape(2, 8, w.S, 3, 256, w.C, 128, quant=quant), "cuda", arena_rows=0, side_arrays=False)
        torch.cuda.synchronize()
        buf.layout(idx, stream=side)
        buf.notify(stream=side)
        buf.notify_expert(idx, stream=side)
        buf.expert_plan(stream=side)
        rows = buf.fp4_rows
        src = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
        weight = torch.full((rows,), -7.0, device="cuda")
        if first_use == "property":
            buf.fp4.q.zero_(), buf.fp4.sf.zero_()
        torch.cuda.synchronize()
        buf.dispatch_expert_fp4(x, idx, weights, stream=side, recv_src_idx=src, recv_weight=weight)
        side.synchronize()
        assert not buf.err.any()
        mine = src >= 0
        got.append((buf.fp4.q.view(rows, -1)[mine], src, weight))
    assert len(got[0][0]) == int((idx >= 0).sum())
    for a, b in zip(*got):
        assert torch.equal(a, b)
