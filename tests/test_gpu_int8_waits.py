"""The int8 product's bounded waits, made to run out without a fault (moe_test_product_wait), and its forms: tiles of each
size, K shared by two pairs, calls at once."""

import threading
import time

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import router_ref as ref
from tests.test_gpu_int8_product import _check, _err, _operands, _plan, _up

pytestmark = pytest.mark.gpu

SHORT = 20_000_000  # cycles: about 10 ms


def _call(E, N, K, gated, operands, rows, plan, y, err):
    moe.moe_expert_product_int8(E, N, K, gated, *operands, rows, plan, y, err)


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("quit_warp", [0, 1, 4, 7, 9, 11])
@pytest.mark.parametrize("form", ["large tiles", "small tiles", "shared K", "shared K, small tiles"])
def test_every_role_ends(form, quit_warp, gated):
    import torch

    if form == "large tiles":
        E, N, K, counts = 6, 4192, 1040, [300, 1, 0, 700, 129, 40]
    elif form == "small tiles":
        E, N, K, counts = 64, 1056, 1040, [2] * 60 + [0, 70, 1, 3]
    else:
        E, N, K, counts = 1, 512, 4112, [300 if form == "shared K" else 60]
    counts = np.array(counts)
    plan, first = _plan(E, counts) if E > 1 else (None, [0, counts[0]])
    rows = int(first[-1])
    operands = _up(*_operands(E, N, K, rows, 1))
    err = _err()
    y = [torch.zeros((rows, N // 2 if gated else N), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    _call(E, N, K, gated, operands, rows, plan, y[0], err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    moe.moe_test_product_wait(SHORT, quit_warp)
    began = time.perf_counter()
    _call(E, N, K, gated, operands, rows, plan, y[1], err)
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 10.0
    assert int(err[0]) == moe.MOE_ERR_DEVICE_TIMEOUT
    err.zero_()
    _call(E, N, K, gated, operands, rows, plan, y[2], err)  # the hook armed one call only
    torch.cuda.synchronize()
    assert int(err[0]) == 0 and torch.equal(y[0], y[2])


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("rows,N,K", [(17, 96, 4096), (60, 512, 4112), (64, 1056, 1040), (65, 288, 2064), (129, 1024, 512),
                                      (200, 4096, 528), (256, 256, 7168), (300, 544, 1552), (513, 2048, 656), (2300, 1120, 400),
                                      (20, 20000 // 32 * 32, 272), (700, 8192, 144)])
def test_dense_calls_of_every_cut(rows, N, K, gated):
    import torch

    wq, ws, xq, xs = _operands(1, N, K, rows, rows + N + K)
    y = torch.full((rows + 1, N // 2 if gated else N), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    _call(1, N, K, gated, _up(wq, ws, xq, xs), rows, None, y, err)
    want, off = ref.product(wq[0], ws[0], xq, xs, gated)
    _check(y[:rows].double().cpu().numpy(), want, off)
    assert (y[rows:] == 7).all() and not err.any()


@pytest.mark.parametrize("counts", [[2] * 250 + [64, 65, 128, 129, 256, 300], [1] * 128, [0] * 127 + [40], [9] * 130])
def test_few_and_many_rows_to_an_expert(counts):
    """Plans whose capacity asks for small tiles, and experts that have more rows than one."""
    import torch

    counts = np.array(counts)
    E, N, K = len(counts), 96, 208
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    wq, ws, xq, xs = _operands(E, N, K, rows, 5)
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    _call(E, N, K, 0, _up(wq, ws, xq, xs), rows, plan, y, err)
    got = y.double().cpu().numpy()
    for e in range(E):
        at = slice(first[e], first[e] + counts[e])
        _check(got[at], *ref.product(wq[e], ws[e], xq[at], xs[at], False), where=e)
        assert (got[first[e] + counts[e]:first[e + 1]] == 7).all()
    assert not err.any()


def test_two_host_threads_and_streams_at_once():
    """Calls of both kernels in flight together, from two threads, give the bits of calls alone."""
    import torch

    cases = [(1, 512, 4112, 1, np.array([300])), (1, 4096, 1040, 0, np.array([5])), (5, 320, 528, 0, np.array([100, 0, 300, 7, 1]))]
    ready, want = [], []
    for E, N, K, gated, counts in cases:
        plan, first = _plan(E, counts) if E > 1 else (None, [0, counts[0]])
        rows = int(first[-1])
        operands = _up(*_operands(E, N, K, rows, N))
        y = torch.zeros((rows, N // 2 if gated else N), dtype=torch.bfloat16, device="cuda")
        _call(E, N, K, gated, operands, rows, plan, y, None)
        ready.append((E, N, K, gated, operands, rows, plan))
        want.append(y)
    torch.cuda.synchronize()
    bad = []

    def work(k):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                for c, w in zip(ready, want):
                    y = torch.zeros_like(w)
                    _call(*c[:4], c[4], *c[5:], y, None)
                    s.synchronize()
                    if not torch.equal(y, w):
                        bad.append((k, c[:4]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_captured_and_replayed_on_changed_inputs():
    import torch

    E, N, K = 3, 256, 1040
    counts = np.array([70, 0, 200])
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    sets = [_up(*_operands(E, N, K, rows, i)) for i in range(2)]
    want = []
    for s in sets:
        y = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
        _call(E, N, K, 0, s, rows, plan, y, None)
        want.append(y)
    held, y = [t.clone() for t in sets[0]], torch.zeros_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(E, N, K, 0, held, rows, plan, y, None)
    for i in (1, 0, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_weights_past_32_bits_of_offset():
    """An expert's weights that start behind the first 2^32 bytes, and rows behind them too."""
    import torch

    E, N, K = 10, 32768, 16384
    counts = np.zeros(E, int)
    counts[-1] = 40
    plan, first = _plan(E, counts)
    w = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    wq, ws, xq, xs = _operands(1, 256, K, 40, 3)
    w[-1, -256:] = torch.from_numpy(wq[0]).cuda()
    scales = torch.zeros((E, N), device="cuda")
    scales[-1, -256:] = torch.from_numpy(ws[0]).cuda()
    y = torch.zeros((40, N), dtype=torch.bfloat16, device="cuda")
    a, b = _up(xq, xs)
    moe.moe_expert_product_int8(E, N, K, 0, w, scales, a, b, 40, plan, y, None)
    _check(y[:, -256:].double().cpu().numpy(), *ref.product(wq[0], ws[0], xq, xs, False))
    assert not y[:, :-256].any()
    # the same rows at the end of slots that pass 2^32 bytes
    stride = 1 << 20
    n = 4200
    rows = torch.zeros((n, stride), dtype=torch.int8, device="cuda")
    rows[-40:, :K] = a
    rows[-40:, K:K + 4] = b.view(torch.int8).view(40, 4)
    one = w[-1, -256:].contiguous()
    out = torch.zeros((n, 256), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_product_int8(1, 256, K, 0, one, scales[-1, -256:].contiguous(), rows, rows.data_ptr() + K, n, None, out, None,
                                x_row_stride=stride, xs_stride=stride)
    assert torch.equal(out[-40:], y[:, -256:])


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("counts,N,K", [([167, 170], 640, 5408), ([254, 0, 300], 64, 4512), ([1], 512, 1040), ([257], 256, 528),
                                        ([33, 31, 64, 65], 96, 272), ([0, 0, 5], 160, 2064), ([600, 2], 288, 1296), ([32, 256], 1056, 144)])
def test_plans_of_few_experts(counts, N, K, gated):
    """Plans whose every tile may have pairs of its own: tiles in parts, and K shared by two to four pairs."""
    import torch

    counts = np.array(counts)
    E = len(counts)
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    wq, ws, xq, xs = _operands(E, N, K, rows, rows + N + K)
    y = torch.full((rows + 1, N // 2 if gated else N), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    _call(E, N, K, gated, _up(wq, ws, xq, xs), rows, plan, y, err)
    got = y.double().cpu().numpy()
    lives = np.zeros(rows + 1, dtype=bool)
    for e in range(E):
        r = slice(int(first[e]), int(first[e]) + int(counts[e]))
        lives[r] = True
        if counts[e]:
            want, off = ref.product(wq[e], ws[e], xq[r], xs[r], gated)
            _check(got[r], want, off)
    assert (got[~lives] == 7).all() and not err.any()


@pytest.mark.parametrize("rows,N,K", [(17, 32, 32768), (32, 512, 7168), (40, 640, 656), (64, 1024, 3088), (120, 256, 1552),
                                      (130, 352, 5472), (250, 416, 3872), (256, 768, 1040), (512, 512, 7168), (30, 32, 384)])
def test_dense_calls_of_which_pairs_share_K(rows, N, K):
    test_dense_calls_of_every_cut(rows, N, K, 0)
    test_dense_calls_of_every_cut(rows, N, K, 1)


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("counts", [[31] * 60 + [130, 256, 257, 700, 0, 1, 128, 129], [700, 513] + [28] * 31 + [128] * 3, [90] * 40,
                                    [0] * 33 + [1500] + [20] * 14])
def test_some_experts_have_far_more_rows_than_the_average(counts, gated):
    """Plans whose average asks for tiles of 128 rows: longer ones are two units each, and a warp looks up 32 at a time."""
    import torch

    counts = np.array(counts)
    E, N, K = len(counts), 288, 400
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    wq, ws, xq, xs = _operands(E, N, K, rows, E)
    y = torch.full((rows, N // 2 if gated else N), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    _call(E, N, K, gated, _up(wq, ws, xq, xs), rows, plan, y, err)
    got = y.double().cpu().numpy()
    for e in range(E):
        at = slice(first[e], first[e] + counts[e])
        if counts[e]:
            _check(got[at], *ref.product(wq[e], ws[e], xq[at], xs[at], gated), where=e)
        assert (got[first[e] + counts[e]:first[e + 1]] == 7).all()
    assert not err.any()


@pytest.mark.parametrize("quit_warp", [0, 1, 4, 7, 9, 11])
def test_every_role_ends_in_tiles_of_128_rows(quit_warp):
    import torch

    counts = np.array([31] * 60 + [130, 256, 257, 700, 0, 1, 128, 129])
    E, N, K = len(counts), 1056, 1040
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    operands = _up(*_operands(E, N, K, rows, 1))
    err = _err()
    y = [torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    _call(E, N, K, 0, operands, rows, plan, y[0], err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    moe.moe_test_product_wait(SHORT, quit_warp)
    _call(E, N, K, 0, operands, rows, plan, y[1], err)
    torch.cuda.synchronize()
    assert int(err[0]) == moe.MOE_ERR_DEVICE_TIMEOUT
    err.zero_()
    _call(E, N, K, 0, operands, rows, plan, y[1], err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0 and torch.equal(y[0], y[1])
