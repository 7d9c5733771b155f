"""What the int8 payload's helpers do on the host, without a GPU."""

import pytest
import torch

from combine_moe_layout_02_gb300 import moe
from tests.test_experts_host import lib, recorder  # noqa: F401  (fixtures)


def _buffers(quant=1, P=2, E=8, S=64, K=2, H=512):
    return moe.Buffers(moe.make_shape(P, E, S, K, H, expert_alignment=128, quant=quant), "cpu", arena_rows=0, side_arrays=False)


@pytest.mark.parametrize("quant", [0, 1])
def test_rows_of_the_4_bit_arena_are_known_with_the_plan(recorder, quant):  # noqa: F811
    """With either payload a caller sizes its arrays by fp4_rows once the plan is made; the rows themselves may come later."""
    buf = _buffers(quant)
    idx, x = torch.zeros((64, 2), dtype=torch.int32), torch.zeros((64, 512), dtype=torch.bfloat16)
    buf.layout(idx)
    buf.notify()
    buf.notify_expert(idx)
    buf.expert_plan()
    rows = buf.fp4_rows
    assert rows % 128 == 0 and rows >= moe.moe_max_expert_rows(buf.shape)
    src, weight = torch.zeros(rows, dtype=torch.int32), torch.zeros(rows)
    buf.dispatch_expert_fp4(x, idx, None, recv_src_idx=src, recv_weight=weight)
    name, args = recorder.calls[-1]
    assert name == "moe_dispatch_expert_fp4" and args[6:9] == (buf.fp4.q.data_ptr(), buf.fp4.sf.data_ptr(), rows)
    assert buf.fp4.rows == rows


def test_rows_of_the_4_bit_arena_may_be_replaced(recorder):  # noqa: F811
    buf = _buffers()
    other = moe.Fp4Rows(buf.fp4_rows, 512, "cpu")
    buf.fp4 = other
    buf.dispatch_expert_fp4(torch.zeros((64, 512), dtype=torch.bfloat16), torch.zeros((64, 2), dtype=torch.int32), None)
    assert buf.fp4 is other and recorder.calls[-1][1][6] == other.q.data_ptr()
