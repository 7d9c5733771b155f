"""The product's long calls: enough work for the order of four row tiles side by side, in every epilogue, at sampled rows.

Two bounds. Element by element that of test_gpu_fp4 (K * 2^-23 * sum |w x|, then bf16). At long rows it is about 4% of
a typical result, so whole rows are held to the norm too: rounding to bf16 is at most 2^-8 of each value, and the sum's
error, some hundred additions each off by 2^-23 of a partial sum of the result's own size, is far below 2^-10 of the
row's norm. A block of 32 that is left out or counted twice is 32 of K terms, sqrt(32 / 7168) = 6.7% of the norm."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import fp4_ref as ref
from tests.test_gpu_experts_large import _dev, _f64, _normal, _tiled_rows

pytestmark = pytest.mark.gpu

TILE_ROWS = 256


def _four_tiles(plan_ints, E, N, K):
    """The launch's rule, from what it knows: the rows that the plan has room for."""
    tiles = (plan_ints - 4 - 2 * (-(-E // 4) * 4)) // 4
    return 2.0 * (tiles - E) * TILE_ROWS * N * K >= 7e12


def _operands(torch, dev, counts, N, K, seed):
    E, first, total = len(counts), [], 0
    for n in counts:
        first.append(total)
        total += -(-n // 128) * 128
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    draw = lambda shape, lo, hi: torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.uint8)
    wt, ch = -(-N // 128), -(-K // 128)
    xq, wq = draw((total, K // 2), 0, 256), draw((E * N, K // 2), 0, 256)
    xsf, wsf = draw((total // 128, ch, 512), 125, 128), draw((E * wt, ch, 512), 120, 123)
    if K % 128:  # scales past the width are 0
        for sf in (xsf, wsf):
            sf.view(-1, ch, 128, 4)[:, -1, :, K % 128 // 32:] = 0
    return first, total, xq, wq, xsf, wsf


@pytest.mark.parametrize("counts,N,K,gated,four", [
    # an odd number of weight tiles, the last of them short, and a last group of fewer than four tiles
    ([30000, 1, 0, 45003, 38000, 9900], 4128, 7168, 0, True),
    ([30000, 1, 0, 45003, 38000, 9900], 4128, 7168, 1, True),
    ([70000, 61003, 300], 7168, 4128, 0, True),  # rows of codes that are no multiple of 128 bytes
    ([900, 3, 0, 1500], 1056, 7168, 0, False),
])
def test_rows_of_long_calls(counts, N, K, gated, four):
    torch, dev = _dev()
    E = len(counts)
    first, total, xq, wq, xsf, wsf = _operands(torch, dev, counts, N, K, N + gated)
    shape = moe.make_shape(1, E, sum(counts), 1, K, expert_alignment=128)
    plan, err = moe.expert_plan_buffer(shape, dev), torch.zeros(4, dtype=torch.int32, device=dev)
    assert _four_tiles(plan.numel(), E, N, K) == four
    assert not four or sum(-(-n // TILE_ROWS) for n in counts) % 4 != 0
    moe.moe_expert_plan(shape, torch.tensor([counts], dtype=torch.int32, device=dev), plan, err)
    back = N // 2 if gated else N
    y = torch.full((total, back), 0x5555, dtype=torch.int16, device=dev)
    moe.moe_expert_product_fp4(E, N, K, gated, wq, wsf, xq, xsf, total, plan, y, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    mine = np.zeros(total, bool)
    for e, (f, n) in enumerate(zip(first, counts)):
        mine[f:f + n] = True
        if n == 0:
            continue
        w = ref.values(ref.unnibble(wq[e * N:(e + 1) * N].cpu().numpy()),
                       ref.untiled(wsf.view(E, -1)[e].cpu().numpy(), N, K))
        at = np.unique(np.concatenate([[f, f + n - 1, f + n // 2], f + np.arange(0, n, max(1, n // 20))]))
        x = ref.values(ref.unnibble(xq[torch.from_numpy(at).to(dev)].cpu().numpy()), _tiled_rows(xsf, total, at, K))
        v, m = x @ w.T, K * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
        if gated:
            i = np.arange(back) // 16 * 32 + np.arange(back) % 16
            gate, up, dg, du = v[:, i], v[:, i + 16], m[:, i], m[:, i + 16]
            with np.errstate(over="ignore"):
                silu = gate / (1 + np.exp(-gate))
            v = silu * up
            m = 1.1 * dg * (np.abs(up) + du) + np.abs(silu) * du + 2.0 ** -18 * np.abs(v)
        tol = m + 2.0 ** -8 * (np.abs(v) + m) + 2.0 ** -126
        got = _f64(y[torch.from_numpy(at).to(dev)])
        assert (np.abs(got - v) <= tol).all(), e
        far = np.linalg.norm(got - v, axis=1) / np.linalg.norm(v, axis=1)
        assert (far <= 2.0 ** -8 + 2.0 ** -10).all(), (e, far.max())
    gap = torch.from_numpy(np.flatnonzero(~mine)).to(dev)
    assert (y[gap] == 0x5555).all()


def test_layer_of_a_long_call():
    """The packing epilogue in that order: the same bits as with the inner rows in bf16, packed by a launch of their own."""
    torch, dev = _dev()
    E, S, K, H, inner = 8, 30000, 4, 7168, 2144
    shape = moe.make_shape(1, E, S, K, H, expert_alignment=128)
    assert 2.0 * (S * K // TILE_ROWS * TILE_ROWS) * 2 * inner * H >= 7e12  # the launch's rule
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    idx = torch.rand((S, E), generator=g, device=dev).argsort(1)[:, :K].to(torch.int32).contiguous()
    wts = torch.rand((S, K), generator=g, device=dev)
    x = _normal(torch, dev, S, H, 1)
    w1 = moe.Fp4Rows(2 * inner, H, dev, groups=E, gated=True).pack(_normal(torch, dev, E * 2 * inner, H, 2))
    w2 = moe.Fp4Rows(H, inner, dev, groups=E).pack(_normal(torch, dev, E * H, inner, 3))
    buf = moe.Buffers(shape, dev, arena_rows=0, side_arrays=False, bits=False)
    args = (x, idx, wts, w1.q.view(E, 2 * inner, -1), w1.sf, w2.q.view(E, H, -1), w2.sf)
    one, two = (torch.full((S, H), v, dtype=torch.int16, device=dev) for v in (1, 2))
    buf.expert_ffn_fp4(*args, one)
    h = torch.zeros((moe.moe_expert_ffn_fp4_rows(shape, inner), inner), dtype=torch.int16, device=dev)
    buf.expert_ffn_fp4(*args, two, h=h)
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    assert torch.equal(one, two)
