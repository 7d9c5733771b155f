"""What the experts' operators do on the host, without a GPU."""

import copy
import glob
import os
import re

import pytest
import torch

from combine_moe_layout_02_gb300 import build as moe_build
from combine_moe_layout_02_gb300 import moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


@pytest.mark.parametrize("cycles,warp", [(0, -1), (1, -2), (1, 12)])
def test_product_wait_hook_refuses(cycles, warp):
    with pytest.raises(moe.MoeError):
        moe.moe_test_product_wait(cycles, warp)


def test_no_load_is_multicast_across_a_cluster():
    """The library takes any device pointer and is loaded by processes that use several GPUs: its loads are plain."""
    sources = glob.glob(os.path.join(os.path.dirname(moe.__file__), "csrc", "*.cu*"))
    assert len(sources) > 10
    for path in sources:
        text = re.sub(r'"\s*"', "", open(path, encoding="utf-8").read())  # adjacent literals are one string
        for line in re.findall(r'"[^"]*cp\.async\.bulk[^"]*"', text):
            assert "multicast" not in line, (path, line)


class _Recorder:
    """Stands in for the library: notes each call's arguments."""

    def __init__(self):
        self.calls = []
        self.real = moe.lib()

    def __getattr__(self, name):
        if not name.startswith("moe_") or name.endswith(("_bytes", "_rows", "_ints")):
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def recorder(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(moe, "lib", lambda: rec)
    monkeypatch.setattr(moe, "_ptr", lambda t: t if t is None or isinstance(t, int) else t.data_ptr())
    monkeypatch.setattr(moe, "_stream", lambda s: s)
    return rec


def _pack_and_unpack(op, rec, rows=3, width=64):
    """(q, sf) of a pack's and an unpack's arguments."""
    x = torch.zeros((rows, width), dtype=torch.bfloat16)
    rec.calls.clear()
    op.pack(x)
    op.unpack(x)
    (a, pack), (b, unpack) = rec.calls
    assert (a, b) == ("moe_fp4_pack", "moe_fp4_unpack") and pack[4] == x.data_ptr() and unpack[6] == x.data_ptr()
    assert pack[:4] == unpack[:4] == (op.groups, op.rows, op.width, int(op.gated))
    return pack[6:8], unpack[4:6]


def test_operand_calls_take_the_tensors_it_holds_now(recorder):
    op = moe.Fp4Rows(3, 64, "cpu")
    assert _pack_and_unpack(op, recorder) == ((op.q.data_ptr(), op.sf.data_ptr()),) * 2
    old = op.q.data_ptr(), op.sf.data_ptr()
    kept = op.q, op.sf  # so that their addresses are not taken again
    op.q, op.sf = torch.zeros_like(op.q), torch.zeros_like(op.sf)
    new = op.q.data_ptr(), op.sf.data_ptr()
    assert new[0] != old[0] and new[1] != old[1] and kept[0].data_ptr() == old[0]
    assert _pack_and_unpack(op, recorder) == (new,) * 2
    op.q.set_(torch.zeros_like(kept[0]))  # other memory under the same tensor
    assert _pack_and_unpack(op, recorder) == ((op.q.data_ptr(), new[1]),) * 2


def test_operand_copies_are_their_own(recorder):
    op = moe.Fp4Rows(3, 64, "cpu")
    op.q.fill_(7)
    twin = copy.deepcopy(op)
    assert twin.q.data_ptr() != op.q.data_ptr() and twin.sf.data_ptr() != op.sf.data_ptr() and (twin.q == 7).all()
    assert _pack_and_unpack(twin, recorder) == ((twin.q.data_ptr(), twin.sf.data_ptr()),) * 2
    assert _pack_and_unpack(op, recorder) == ((op.q.data_ptr(), op.sf.data_ptr()),) * 2


def test_operand_refuses_other_tensors_in_its_place(recorder):
    op = moe.Fp4Rows(3, 64, "cpu", groups=2)
    for bad in (torch.zeros_like(op.q, dtype=torch.int8), torch.zeros(op.q.numel() - 1, dtype=torch.uint8),
                torch.zeros((6, 64), dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError):
            op.q = bad
    with pytest.raises(ValueError):
        op.sf = torch.zeros(512, dtype=torch.uint8)


def test_operand_refuses_rows_of_another_type_or_size(recorder):
    op = moe.Fp4Rows(3, 64, "cpu", groups=2)
    for call in (op.pack, op.unpack):
        for bad in (torch.zeros((6, 64)), torch.zeros((6, 64), dtype=torch.float16), torch.zeros((5, 64), dtype=torch.bfloat16),
                    torch.zeros((6, 96), dtype=torch.bfloat16), torch.zeros((6, 32), dtype=torch.bfloat16)):
            with pytest.raises(ValueError):
                call(bad)
        assert not recorder.calls
        call(torch.zeros((2, 3, 64), dtype=torch.int16))
        call(torch.zeros((8, 64), dtype=torch.bfloat16))  # rows to spare
        recorder.calls.clear()
