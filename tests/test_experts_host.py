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
        if not name.startswith("moe_") or name.endswith(("_bytes", "_rows", "_ints", "_stride", "_string")):
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


def _layer(E=4, S=6, K=2, H=64, inner=96):
    """Buffers without a GPU, and a layer call's arguments by name."""
    buf = moe.Buffers.__new__(moe.Buffers)
    buf.shape, buf.device, buf.err = moe.make_shape(1, E, S, K, H), "cpu", torch.zeros(4, dtype=torch.int32)
    sizes = (E * inner * H, E * moe.moe_fp4_scale_bytes(2 * inner, H), E * H * inner // 2, E * moe.moe_fp4_scale_bytes(H, inner))
    buf._ffn_workspaces = {inner: (torch.zeros(64, dtype=torch.uint8), {0})}
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    args = dict(x=torch.zeros((S, H), dtype=torch.bfloat16), topk_idx=torch.zeros((S, K), dtype=torch.int32),
                topk_weights=torch.zeros((S, K)), w1=u8(E, 2 * inner, H // 2), w1_sf=u8(sizes[1]), w2=u8(E, H, inner // 2),
                w2_sf=u8(sizes[3]), out=torch.zeros((S, H), dtype=torch.bfloat16))
    return buf, args, inner


def test_layer_refuses_tensors_that_are_not_its_own(recorder):
    buf, args, inner = _layer()
    call = lambda **k: buf.expert_ffn_fp4(**{**args, **k}, stream=0)
    call()
    call(topk_weights=None)
    call(x=args["x"].view(torch.int16), out=torch.zeros((9, 64), dtype=torch.int16))  # rows to spare
    call(w1=args["w1"].reshape(-1), w2=args["w2"].view(-1, inner // 2))
    call(h=torch.zeros((moe.moe_expert_ffn_fp4_rows(buf.shape, inner), inner), dtype=torch.bfloat16))
    assert [n for n, _ in recorder.calls] == ["moe_expert_ffn_fp4"] * 5
    recorder.calls.clear()
    half = lambda t: t.reshape(-1)[: t.numel() // 2]
    bad = [dict(w1=args["w1"][:, : inner]), dict(w1=args["w1"][:3]), dict(w1_sf=half(args["w1_sf"])),
           dict(w2_sf=half(args["w2_sf"])), dict(w2=args["w2"][:3]), dict(w1=torch.zeros((4, 2 * inner, 64), dtype=torch.uint8)),
           dict(w1=args["w1"].to(torch.bfloat16)), dict(x=args["x"].float()), dict(x=args["x"][:5]),
           dict(x=torch.zeros((6, 96), dtype=torch.bfloat16)), dict(x=args["x"].half()), dict(out=args["out"].float()),
           dict(out=args["out"][:5]), dict(topk_idx=args["topk_idx"].long()), dict(topk_idx=args["topk_idx"][:, :1]),
           dict(topk_weights=args["topk_weights"].bfloat16()), dict(topk_weights=args["topk_weights"][:3]),
           dict(h=torch.zeros((6, inner), dtype=torch.bfloat16))]
    for k in bad:
        with pytest.raises(ValueError):
            call(**k)
    for k in (dict(w2=torch.zeros((4, 64, 24), dtype=torch.uint8)), dict(w2=torch.zeros((4, 64, 0), dtype=torch.uint8))):
        with pytest.raises(moe.MoeError):  # no inner width
            call(**k)
    assert not recorder.calls and list(buf._ffn_workspaces) == [inner]  # nothing was made for what is refused


def _fp4_path(buf, idx, x):
    buf.layout(idx)
    buf.notify()
    buf.notify_expert(idx)
    buf.expert_plan()
    buf.dispatch_expert_fp4(x, idx, None)


def test_the_4_bit_path_makes_no_bf16_arena(recorder, monkeypatch):
    """notify_expert makes the tables of the slots; the arena comes with the calls that use it."""
    P, E, S, K, H = 2, 8, 64, 2, 512
    shape = moe.make_shape(P, E, S, K, H, expert_alignment=128)
    arena = moe.moe_max_expert_rows(shape) * moe.moe_slot_stride(H, 0)
    made, real = [], torch.empty

    def empty(*args, **kw):
        t = real(*args, **kw)
        made.append(t.nbytes)
        return t

    monkeypatch.setattr(torch, "empty", empty)
    buf = moe.Buffers(shape, "cpu", arena_rows=0, side_arrays=False)
    idx, x = torch.zeros((S, K), dtype=torch.int32), torch.zeros((S, H), dtype=torch.bfloat16)
    _fp4_path(buf, idx, x)
    assert max(made) < arena // 2
    buf.dispatch_expert(x, idx, None)
    assert max(made) == arena
    name, args = recorder.calls[-1]
    assert name == "moe_dispatch_expert" and args[6] == buf.expert_arena.data_ptr() and args[7] == buf.expert_rows
    assert args[8:10] == (buf.expert_src_idx.data_ptr(), buf.expert_weight.data_ptr())


@pytest.mark.parametrize("arena_rows", [None, 0])
def test_combine_reads_the_rows_that_it_is_given(recorder, arena_rows):
    P, E, S, K, H = 2, 8, 64, 2, 512
    buf = moe.Buffers(moe.make_shape(P, E, S, K, H, expert_alignment=128), "cpu", arena_rows=0, side_arrays=False)
    idx, x = torch.zeros((S, K), dtype=torch.int32), torch.zeros((S, H), dtype=torch.bfloat16)
    buf.layout(idx)
    buf.notify()
    buf.notify_expert(idx, arena_rows=arena_rows)
    buf.expert_plan()
    buf.dispatch_expert_fp4(x, idx, None)
    rows_of = lambda: recorder.calls[-1][1][4]
    out = torch.empty_like(x)
    buf.combine_expert(out, idx, None, y=torch.zeros((buf.fp4_rows, H), dtype=torch.bfloat16), y_row_stride=2 * H)
    assert recorder.calls[-1][0] == "moe_combine_expert" and rows_of() == buf.fp4_rows
    buf.combine_expert(out, idx, None, y=torch.zeros((100, H + 8), dtype=torch.bfloat16), y_row_stride=2 * H + 16)
    assert rows_of() == 100
    buf.combine_expert(out, idx, None, y=torch.zeros(100 * (H + 8) - 8, dtype=torch.bfloat16), y_row_stride=2 * H + 16)
    assert rows_of() == 100  # the last row ends where the tensor does
    buf.combine_expert(out, idx, None, y=torch.zeros(0, dtype=torch.bfloat16), y_row_stride=2 * H)
    assert rows_of() == 0
    buf.combine_expert(out, idx, None, y=1 << 20, y_row_stride=2 * H)  # an address: as many as the arena's
    assert rows_of() == (moe.moe_max_expert_rows(buf.shape) if arena_rows is None else arena_rows)


def test_an_arena_of_the_programs_own(recorder):
    """The arena and its side arrays may be replaced, before they are made as well."""
    buf = moe.Buffers(moe.make_shape(2, 8, 64, 2, 64), "cpu", arena_rows=0, side_arrays=False)
    idx, x = torch.zeros((64, 2), dtype=torch.int32), torch.zeros((64, 64), dtype=torch.bfloat16)
    buf.notify_expert(idx)
    arena = buf.expert_arena = torch.zeros((buf.expert_rows, buf.stride), dtype=torch.uint8)
    buf.dispatch_expert(x, idx, None)
    assert recorder.calls[-1][1][6] == arena.data_ptr() and buf.expert_arena is arena
    assert recorder.calls[-1][1][8] == buf.expert_src_idx.data_ptr()
    weight = buf.expert_weight = torch.zeros(buf.expert_rows)
    buf.dispatch_expert(x, idx, None)
    assert recorder.calls[-1][1][9] == weight.data_ptr()
