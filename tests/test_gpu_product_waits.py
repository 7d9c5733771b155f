"""The product's bounded waits, made to run out without a fault: a warp of each CTA acts as if its first wait had run out
(moe_test_product_wait). Every role then ends, the error word says so, and the next call on the same buffers gives the
same bits as before."""

import time

import pytest

from combine_moe_layout_02_gb300 import inputs, moe
from tests.test_gpu_fp4 import _rows, _up

pytestmark = pytest.mark.gpu

SHORT = 20_000_000  # cycles: about 10 ms


def _layer(E, S, K, H, inner, seed):
    import torch

    dev = torch.device("cuda", 0)
    w = inputs.make(1, E, S, H, K, seed=seed, expert_alignment=128)
    w1 = moe.Fp4Rows(2 * inner, H, dev, groups=E, gated=True).pack(_up(_rows(E * 2 * inner, H, 1)))
    w2 = moe.Fp4Rows(H, inner, dev, groups=E).pack(_up(_rows(E * H, inner, 2)))
    buf = moe.Buffers(moe.make_shape(1, E, S, K, H, expert_alignment=128), dev, arena_rows=0, side_arrays=False)
    idx, wts = torch.from_numpy(w.topk_idx).to(dev), torch.from_numpy(w.topk_weights).to(dev)
    args = (_up(w.x_bits), idx, wts, w1.q.view(E, 2 * inner, -1), w1.sf, w2.q.view(E, H, -1), w2.sf)
    return buf, args


@pytest.mark.parametrize("quit_warp", [0, 1, 4, 6, 7, 9, 11])
def test_the_packing_epilogue_ends_together(quit_warp):
    """A warp of a group of four gives up while the others' sums are complete: nobody is left at the group's barrier."""
    import torch

    # several units per CTA, more stages than the ring holds
    buf, args = _layer(16, 1500, 4, 2080, 608, seed=3)
    out = [torch.zeros((1500, 2080), dtype=torch.int16, device="cuda") for _ in range(3)]
    buf.expert_ffn_fp4(*args, out[0])
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    moe.moe_test_product_wait(SHORT, quit_warp)
    began = time.perf_counter()
    buf.expert_ffn_fp4(*args, out[1])
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 10.0
    assert int(buf.err[0]) == moe.MOE_ERR_DEVICE_TIMEOUT
    buf.err.zero_()
    buf.expert_ffn_fp4(*args, out[2])  # the hook armed one call only
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    assert torch.equal(out[0], out[2])


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("quit_warp", [0, 1, 5, 10])
def test_the_other_epilogues_end(gated, quit_warp):
    import torch

    dev = torch.device("cuda", 0)
    E, N, K, counts = 6, 1056, 2080, [300, 1, 0, 700, 129, 40]
    total = sum(-(-n // 128) * 128 for n in counts)
    shape = moe.make_shape(1, E, sum(counts), 1, K, expert_alignment=128)
    plan, err = moe.expert_plan_buffer(shape, dev), torch.zeros(4, dtype=torch.int32, device=dev)
    moe.moe_expert_plan(shape, torch.tensor([counts], dtype=torch.int32, device=dev), plan, err)
    w = moe.Fp4Rows(N, K, dev, groups=E).pack(_up(_rows(E * N, K, 1)))
    x = moe.Fp4Rows(total, K, dev).pack(_up(_rows(total, K, 2)))
    y = [torch.zeros((total, N // 2 if gated else N), dtype=torch.int16, device=dev) for _ in range(3)]
    call = lambda out: moe.moe_expert_product_fp4(E, N, K, gated, w.q, w.sf, x.q, x.sf, total, plan, out, err)
    call(y[0])
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    moe.moe_test_product_wait(SHORT, quit_warp)
    began = time.perf_counter()
    call(y[1])
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 10.0
    assert int(err[0]) == moe.MOE_ERR_DEVICE_TIMEOUT
    err.zero_()
    call(y[2])
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    assert torch.equal(y[0], y[2])
