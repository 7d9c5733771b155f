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


A = 1 << 20  # an aligned address, never read


def _product(**k):
    """A call whose other arguments are addresses: what is refused is the tensor that is given."""
    a = {**dict(wq=A, ws=A, xq=A, xs=A, y=A, plan=None, err=None, E=1, gated=0), **k}
    moe.moe_expert_product_int8(a["E"], 64, 32, a["gated"], a["wq"], a["ws"], a["xq"], a["xs"], 5, a["plan"], a["y"], a["err"])


def test_packed_rows_have_their_width():
    """A larger tensor whose rows are wider would be read, or written, at the wrong places."""
    i8, bf = lambda *s: torch.zeros(s, dtype=torch.int8), lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for bad in (dict(wq=i8(1, 64, 48)), dict(wq=i8(128, 64)), dict(xq=i8(5, 48)), dict(xq=i8(10, 16)), dict(y=bf(5, 128)),
                dict(y=bf(10, 32)), dict(y=bf(5, 64), gated=1)):
        with pytest.raises(ValueError, match="with rows of"):
            _product(**bad)
    for good in (dict(wq=i8(1, 64, 32)), dict(wq=i8(64 * 32)), dict(xq=i8(7, 32)), dict(y=bf(5, 64)), dict(y=bf(320)),
                 dict(y=bf(5, 32), gated=1)):
        with pytest.raises(ValueError, match="CUDA"):  # nothing but its place is wrong
            _product(**good)


def test_plans_and_error_words_are_held_to_their_type_and_place():
    for bad in (dict(E=2, plan=torch.zeros(64, dtype=torch.int64)), dict(E=2, plan=torch.zeros(64)), dict(err=torch.zeros(4)),
                dict(E=2, plan=torch.zeros((64, 2), dtype=torch.int32)[:, 0]), dict(err=torch.zeros(0, dtype=torch.int32))):
        with pytest.raises(ValueError, match="expected (plan|err)"):
            _product(**bad)
    for bad in (dict(E=2, plan=torch.zeros(64, dtype=torch.int32)), dict(err=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            _product(**bad)


def test_packing_holds_its_plan():
    op = moe.Int8Rows(4, 64, "cpu")
    with pytest.raises(ValueError):
        op.pack(torch.zeros((4, 64), dtype=torch.bfloat16), E=2, plan=torch.zeros(64, dtype=torch.int64))


def test_a_plan_s_experts_may_be_any_whole_number(monkeypatch):
    """As the other calls that take a plan: a count out of numpy will do."""
    import numpy as np

    plan = torch.zeros(64, dtype=torch.int32)
    monkeypatch.setattr(moe, "_flat", lambda t, n, dtype, name: t.data_ptr())
    for e, _, ints in (moe._plan_on(np.int64(2), plan, 0), moe._plan_on(np.int64(2), plan, plan.get_device())):
        assert type(e) is int and e == 2 and ints == 64
