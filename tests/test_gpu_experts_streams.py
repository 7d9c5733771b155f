"""The expert layer's memory on several streams: workspaces that calls in flight use go to nobody else; two host threads
with a layer each; a captured layer replayed on changed inputs."""

import threading

import pytest

from combine_moe_layout_02_gb300 import inputs, moe
from tests.test_gpu_fp4 import _rows, _up

pytestmark = pytest.mark.gpu

E, K, H = 8, 2, 256


def _weights(inner, seed):
    import torch

    dev = torch.device("cuda", 0)
    w1 = moe.Fp4Rows(2 * inner, H, dev, groups=E, gated=True).pack(_up(_rows(E * 2 * inner, H, seed)))
    w2 = moe.Fp4Rows(H, inner, dev, groups=E).pack(_up(_rows(E * H, inner, seed + 1)))
    return w1.q.view(E, 2 * inner, -1), w1.sf, w2.q.view(E, H, -1), w2.sf


def _batch(S, seed):
    import torch

    w = inputs.make(1, E, S, H, K, seed=seed, expert_alignment=128)
    dev = torch.device("cuda", 0)
    return _up(w.x_bits), torch.from_numpy(w.topk_idx).to(dev), torch.from_numpy(w.topk_weights).to(dev)


def _buffers(S):
    return moe.Buffers(moe.make_shape(1, E, S, K, H), "cuda", arena_rows=0, side_arrays=False, bits=False)


def test_a_workspace_outlives_calls_of_another_width():
    """Two layers of different widths on the same buffers: neither's memory goes back while the other is called."""
    import torch

    S = 200
    buf, batch = _buffers(S), _batch(S, 1)
    narrow, wide = _weights(64, 1), _weights(608, 2)
    out = torch.empty_like(batch[0])
    used, real = [], moe.moe_expert_ffn_fp4

    def noted(*args):
        used.append((args[10].data_ptr(), args[10].numel()))
        return real(*args)

    moe.moe_expert_ffn_fp4 = noted
    try:
        for w in (narrow, wide, narrow, wide):
            buf.expert_ffn_fp4(*batch, *w, out)
            torch.cuda.synchronize()
            taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in used for _ in range(4)]
            for t in taken:
                assert all(t.data_ptr() + t.numel() <= p or t.data_ptr() >= p + n for p, n in used)
            del taken
    finally:
        moe.moe_expert_ffn_fp4 = real
    assert used[0] == used[2] and used[1] == used[3] and used[0] != used[1]
    assert int(buf.err[0]) == 0


def test_a_workspace_waits_for_the_streams_that_use_it():
    """Buffers dropped while a call of theirs is queued on a side stream: its workspace is not handed out before."""
    import torch

    S = 200
    batch, w = _batch(S, 1), _weights(608, 2)
    out = torch.empty_like(batch[0])
    want = torch.empty_like(out)
    _buffers(S).expert_ffn_fp4(*batch, *w, want)
    torch.cuda.synchronize()
    for how in ("argument", "current"):
        side = torch.cuda.Stream()
        buf = _buffers(S)
        n = moe.moe_expert_ffn_fp4_workspace_bytes(buf.shape, 608)
        # memory and kernels at hand: an allocation from the driver, or a kernel's first use, waits for the device
        spare = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(6)]
        del spare
        err, seen, real = buf.err, [], moe.moe_expert_ffn_fp4

        def noted(*args):
            seen.append((args[10].data_ptr(), args[10].numel()))
            return real(*args)

        moe.moe_expert_ffn_fp4 = noted
        try:
            buf.expert_ffn_fp4(*batch, *w, out)  # on the default stream first
            torch.cuda.synchronize()
            out.zero_()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(100_000_000)  # about 50 ms
                if how == "current":
                    buf.expert_ffn_fp4(*batch, *w, out)
            if how == "argument":
                buf.expert_ffn_fp4(*batch, *w, out, stream=side)
        finally:
            moe.moe_expert_ffn_fp4 = real
        assert seen[0] == seen[1] and seen[0][1] == n and not side.query()
        del buf
        taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.current_stream().synchronize()
        assert not side.query(), "the side stream was done too early for this test to see anything"
        assert all(t.data_ptr() + n <= seen[0][0] or t.data_ptr() >= seen[0][0] + n for t in taken)
        side.synchronize()
        assert int(err[0]) == 0 and torch.equal(out, want)
        del taken


def test_a_workspace_is_made_on_the_stream_that_uses_it():
    """The first call on a side stream does not write memory that the current stream's queued work still reads."""
    import torch

    S = 200
    batch, w = _batch(S, 1), _weights(608, 2)
    out = torch.empty_like(batch[0])
    side = torch.cuda.Stream()
    buf = _buffers(S)
    n = moe.moe_expert_ffn_fp4_workspace_bytes(buf.shape, 608)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full((n,), 0x2A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    still = old.clone()  # queued behind the sleep: reads `old` then
    del old
    buf.expert_ffn_fp4(*batch, *w, out, stream=side)
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    assert (still == 0x2A).all()


def test_threads_with_a_layer_each():
    import torch

    sizes = [(64, 300), (160, 77), (608, 1200), (32, 9)]
    want, jobs = [], []
    for i, (inner, S) in enumerate(sizes):
        batch, w = _batch(S, 10 + i), _weights(inner, 20 + i)
        out = torch.empty_like(batch[0])
        _buffers(S).expert_ffn_fp4(*batch, *w, out)
        want.append(out)
        jobs.append((S, batch, w))
    torch.cuda.synchronize()
    got, start = [None] * len(jobs), threading.Barrier(len(jobs))

    def work(i):
        try:
            S, batch, w = jobs[i]
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                buf, out = _buffers(S), torch.empty_like(batch[0])
            start.wait()
            for _ in range(25):
                buf.expert_ffn_fp4(*batch, *w, out, stream=st)
            st.synchronize()
            got[i] = out, int(buf.err[0])
        except BaseException as e:  # reported by the main thread
            got[i] = e

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
        assert not t.is_alive()
    for a, b in zip(got, want):
        if isinstance(a, BaseException):
            raise a
        assert a[1] == 0 and torch.equal(a[0], b)


def test_a_captured_layer_on_changed_inputs():
    """One capture; replayed after the batch's rows, routing and weights were replaced in place."""
    import torch

    S, inner = 500, 160
    buf, w = _buffers(S), _weights(inner, 3)
    x, idx, wts = (t.clone() for t in _batch(S, 1))
    out = torch.empty_like(x)
    buf.expert_ffn_fp4(x, idx, wts, *w, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.expert_ffn_fp4(x, idx, wts, *w, out)
    for seed in (1, 2, 3):
        for t, v in zip((x, idx, wts), _batch(S, seed)):
            t.copy_(v)
        if seed == 3:
            idx[::5] = -1
        out.fill_(0x5555)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        fresh = _buffers(S)
        fresh.expert_ffn_fp4(x, idx, wts, *w, out)
        torch.cuda.synchronize()
        assert int(buf.err[0]) == 0 and int(fresh.err[0]) == 0
        assert torch.equal(got, out)


def test_the_4_bit_path_by_its_public_methods():
    """Step by step without a bf16 arena: the layer's own bits, combine reading the down product's rows."""
    import torch

    S, inner, P = 640, 160, 4
    shape = moe.make_shape(P, E, S, K, H, expert_alignment=128)
    (x, idx, wts), (w1, w1sf, w2, w2sf) = _batch(S, 5), _weights(inner, 7)
    want = torch.empty_like(x)
    _buffers(S).expert_ffn_fp4(x, idx, wts, w1, w1sf, w2, w2sf, want)
    buf = moe.Buffers(shape, "cuda", arena_rows=0, side_arrays=False, bits=False)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    buf.layout(idx)
    buf.notify()
    buf.notify_expert(idx)
    buf.expert_plan()
    buf.dispatch_expert_fp4(x, idx, wts)
    assert torch.cuda.max_memory_allocated() - before < moe.moe_max_expert_rows(shape) * moe.moe_slot_stride(H, 0)
    rows = buf.fp4_rows
    h, y, out = (torch.zeros((n, m), dtype=torch.int16, device="cuda") for n, m in ((rows, inner), (rows, H), (S, H)))
    moe.moe_expert_product_fp4(E, 2 * inner, H, 1, w1, w1sf, buf.fp4.q, buf.fp4.sf, rows, buf.plan, h, buf.err)
    hq = moe.Fp4Rows(rows, inner).pack(h, E, buf.plan)
    moe.moe_expert_product_fp4(E, H, inner, 0, w2, w2sf, hq.q, hq.sf, rows, buf.plan, y, buf.err)
    buf.combine_expert(out, idx, wts, y=y, y_row_stride=2 * H)
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("what", ["fp4", "arena"])
def test_first_calls_make_their_memory_on_their_stream(what):
    """As the workspace: operands and arenas that a first call makes on a side stream."""
    import torch

    S = 4000
    x, idx, wts = _batch(S, 1)
    side = torch.cuda.Stream()
    buf = moe.Buffers(moe.make_shape(1, E, S, K, H, expert_alignment=128), "cuda", arena_rows=0, side_arrays=False)
    rows = (moe.moe_max_expert_rows(buf.shape) + 127) // 128 * 128
    n = rows * (H // 2) if what == "fp4" else moe.moe_max_expert_rows(buf.shape) * buf.stride

    def calls(b):
        b.notify_expert(idx, stream=side)
        if what == "fp4":
            b.expert_plan(stream=side)
            b.dispatch_expert_fp4(x, idx, wts, stream=side)
        else:
            b.dispatch_expert(x, idx, wts, stream=side)

    first = moe.Buffers(buf.shape, "cuda", arena_rows=0, side_arrays=False)
    for b in (first, buf):
        b.layout(idx)
        b.notify()
    calls(first)  # a kernel's first use waits for the device
    torch.cuda.synchronize()
    del b, first
    torch.cuda.empty_cache()
    old = torch.full((n,), 0x2A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    still = old.clone()  # queued behind the sleep: reads `old` then
    del old
    calls(buf)
    assert (buf.fp4.q if what == "fp4" else buf.expert_arena).nbytes == n
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    assert (still == 0x2A).all()


@pytest.mark.parametrize("how", ["handle", "external", "current"])
def test_a_stream_that_is_not_torchs_may_go_first(how):
    """A stream made and destroyed by the program itself: buffers that were used on it are dropped afterwards."""
    import ctypes
    import gc

    import torch

    cuda = moe.lib()  # finds the CUDA runtime that the library is linked to
    cuda.cudaStreamCreateWithFlags.argtypes = [ctypes.c_void_p, ctypes.c_uint]
    cuda.cudaStreamDestroy.argtypes = cuda.cudaStreamSynchronize.argtypes = [ctypes.c_void_p]
    S = 200
    batch, w = _batch(S, 1), _weights(608, 2)
    want, out = torch.empty_like(batch[0]), torch.empty_like(batch[0])
    buf = _buffers(S)
    buf.expert_ffn_fp4(*batch, *w, want)  # torch's own stream first
    torch.cuda.synchronize()
    raw = ctypes.c_void_p()
    assert cuda.cudaStreamCreateWithFlags(ctypes.byref(raw), 1) == 0
    for _ in range(2):
        out.zero_()
        torch.cuda.synchronize()
        if how == "handle":
            buf.expert_ffn_fp4(*batch, *w, out, stream=raw.value)
        elif how == "external":
            buf.expert_ffn_fp4(*batch, *w, out, stream=torch.cuda.ExternalStream(raw.value))
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(raw.value)):
                buf.expert_ffn_fp4(*batch, *w, out)
        assert cuda.cudaStreamSynchronize(raw) == 0
        assert torch.equal(out, want)
    assert int(buf.err[0]) == 0
    assert cuda.cudaStreamDestroy(raw) == 0
    del buf
    gc.collect()
    again = _buffers(S)
    again.expert_ffn_fp4(*batch, *w, out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
