"""The int8 product in a steady state: every pair of CTAs has many units, stages go round the ring many times, and the whole
result is compared with whole-number sums formed on the GPU."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests.test_gpu_int8_product import BF, _err, _plan

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23


def _codes(shape, g):
    import torch

    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        part = flat[a:a + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127))
    return out


def _whole_sums(x, w):
    """x [rows, K] . w [N, K] of codes, exact: 1024 products of codes stay below 2^24, which binary32 holds, and 64 bits add."""
    import torch

    v = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 1024):
        v += x[:, k:k + 1024].float() @ w[:, k:k + 1024].float().T
    return v


def _wanted(x, w, ws, xs, gated):
    """The result in 64 bits, and what it may be off by before it is rounded to bf16."""
    import torch

    # Sums below 2^24 on the way in any order (Cauchy and Schwarz), so binary32 sums are exact; then two products.
    norm = lambda t: (t.float() ** 2).sum(1).max().sqrt()
    assert float(norm(x) * norm(w)) < 2 ** 24
    v = _whole_sums(x, w) * ws.double() * xs.double()[:, None]
    off = v.abs() * ULP
    if not gated:
        return v, off
    at = torch.arange(v.shape[1] // 2, device="cuda")
    at = at // 16 * 32 + at % 16
    g, u = v[:, at], v[:, at + 16]
    silu = g * torch.sigmoid(g)
    # the exponential's 2 + 1.173 |g| units, a sum, a quotient (2 units) and two products; silu's slope is below 1.1
    y = silu * u
    return y, y.abs() * (2 + 1.173 * g.abs() + 6) * ULP + 1.1 * off[:, at] * u.abs() + silu.abs() * off[:, at + 16]


def _check_all(E, N, K, counts, gated, slots, repeats, seed=0):
    import torch

    assert not torch.backends.cuda.matmul.allow_tf32
    g = torch.Generator(device="cuda").manual_seed(seed)
    plan, first = _plan(E, counts)
    rows, width = int(first[-1]), N // 2 if gated else N
    stride, at = (moe.moe_slot_stride(K, 1), (K + 31) // 32 * 32) if slots else (K, 0)
    err = _err()
    for turn in range(repeats):
        wq, ws = _codes((E, N, K), g), (torch.rand((E, N), generator=g, device="cuda") + 0.5) / (32 * K ** 0.5)
        xq, xs = _codes((rows, K), g), (torch.rand((rows,), generator=g, device="cuda") + 0.5) / 32
        x, s, kw = xq, xs, {}
        if slots:
            x = torch.full((rows, stride), 7, dtype=torch.int8, device="cuda")
            x[:, :K] = xq
            x[:, at:at + 4] = xs.view(torch.int8).view(rows, 4)
            s, kw = x.data_ptr() + at, dict(x_row_stride=stride, xs_stride=stride)
        y = [torch.full((rows, width), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for out in y:
            moe.moe_expert_product_int8(E, N, K, gated, wq, ws, x, s, rows, plan, out, err, **kw)
        assert torch.equal(y[0].view(torch.int16), y[1].view(torch.int16)), turn
        for e in range(E):
            r = slice(int(first[e]), int(first[e] + counts[e]))
            if counts[e]:
                want, off = _wanted(xq[r], wq[e], ws[e], xs[r], gated)
                bad = (y[0][r].double() - want).abs() > want.abs() * BF + off * (1 + BF) + 1e-38
                assert not bad.any(), (turn, e, int(bad.sum()), bad.nonzero()[:4].tolist())
            assert (y[0][int(first[e] + counts[e]):int(first[e + 1])] == 7).all()
    assert not err.any()


def _counts(E, least, most, seed):
    return np.random.default_rng(seed).integers(least, most + 1, E)


@pytest.mark.parametrize("E,N,K,least,most,gated,slots,repeats", [
    (64, 4096, 7168, 500, 1100, 1, True, 24),   # tiles of 256 rows, weights out of HBM
    (64, 7168, 2048, 500, 1100, 0, False, 24),
    (16, 1024, 4096, 900, 2300, 0, True, 24),   # weights that L2 holds
    (64, 1024, 1024, 30, 150, 0, True, 24),     # tiles of 128 rows
    (64, 2048, 2048, 30, 90, 1, False, 12),
    (128, 1024, 512, 1, 40, 0, False, 24),      # tiles of 64 rows
    (64, 1024, 1536, 0, 30, 1, True, 24),
])
def test_the_whole_result(E, N, K, least, most, gated, slots, repeats):
    _check_all(E, N, K, _counts(E, least, most, E + N), gated, slots, repeats, seed=K)


@pytest.mark.parametrize("K", [16, 64, 160, 192, 416, 448])
@pytest.mark.parametrize("gated", [0, 1])
def test_short_ends_of_k_in_tiles_of_128_rows(K, gated):
    """K of one, two and four stages whose last has one half: a converting group waits for no product there."""
    _check_all(256, 1024, K, _counts(256, 25, 110, K), gated, bool(gated), 30, seed=K)
