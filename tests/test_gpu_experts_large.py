"""The experts' operators where byte offsets and element counts pass 32 bits, checked at sampled rows
(the first, the last and some between) against the 64-bit definitions."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import fp4_ref as ref
from tests.helpers import bf16_bits_to_f32, f32_to_bf16_bits_torch

pytestmark = pytest.mark.gpu


def _dev():
    import torch

    return torch, torch.device("cuda", 0)


def _f64(t):
    return bf16_bits_to_f32(t.cpu().numpy().view(np.uint16)).astype(np.float64)


def _normal(torch, dev, rows, width, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.empty((rows, width), dtype=torch.bfloat16, device=dev)
    for a in range(0, rows, 65536):
        x[a:a + 65536].normal_(generator=g)
    return x.view(torch.int16)


def _some(rows, n=40, seed=0):
    return np.unique(np.concatenate([[0, rows - 1], np.random.default_rng(seed).integers(0, rows, n)]))


def test_pack_and_unpack():
    torch, dev = _dev()
    rows, width = 620_001, 7168  # 4.4e9 elements
    x = _normal(torch, dev, rows, width, 1)
    op = moe.Fp4Rows(rows, width, dev).pack(x)
    back = torch.empty_like(x)
    op.unpack(back)
    at = _some(rows)
    pick = torch.from_numpy(at).to(dev)
    codes, s = ref.pack(_f64(x[pick]))
    np.testing.assert_array_equal(op.q[pick].cpu().numpy(), ref.nibbles(codes))
    sf = op.sf.view(-1, width // 128, 512)[pick // 128].cpu().numpy()
    for i, m in enumerate(at):
        o = m % 32 * 16 + m % 128 // 32 * 4
        np.testing.assert_array_equal(sf[i, :, o:o + 4].reshape(-1), s[i])
    np.testing.assert_array_equal(_f64(back[pick]), ref.values(codes, s))


def test_dispatch_and_product():
    """1.28 million rows of 7168 (4.6 GB of codes): rows of the last expert come out as those of the first."""
    torch, dev = _dev()
    P, E, S, K, H, N = 4, 8, 160_000, 8, 7168, 32
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    x = _normal(torch, dev, S, H, 3)
    idx = torch.rand((S, E), generator=g, device=dev).argsort(1)[:, :K].to(torch.int32).contiguous()
    shape = moe.make_shape(P, E, S, K, H, expert_alignment=128)
    buf = moe.Buffers(shape, dev, arena_rows=0, side_arrays=False, bits=False)
    buf.layout(idx)
    buf.notify()
    buf._fp4_buffers()
    moe.moe_notify_expert(shape, idx, buf.num_recv_tokens_per_expert, buf.recv_expert_offset, buf.slot_row,
                          buf.expert_part_base, buf.scratch)
    buf.expert_plan()
    buf.dispatch_expert_fp4(x, idx, None)
    assert buf.fp4.q.numel() > 2 ** 32
    w = moe.Fp4Rows(N, H, dev, groups=E).pack(_normal(torch, dev, E * N, H, 4))
    y = torch.full((buf.fp4_rows, N), 0x5555, dtype=torch.int16, device=dev)
    moe.moe_expert_product_fp4(E, N, H, 0, w.q, w.sf, buf.fp4.q, buf.fp4.sf, buf.fp4_rows, buf.plan, y, buf.err)
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    wv = ref.values(ref.unnibble(w.q.cpu().numpy()), np.concatenate(
        [ref.untiled(p, N, H) for p in w.sf.cpu().numpy().reshape(E, -1)])).reshape(E, N, H)
    base = buf.expert_part_base.cpu().numpy()
    last = 0
    for t in _some(S, 60):
        codes, s = ref.pack(_f64(x[t:t + 1]))
        xv = ref.values(codes, s)[0]
        for k in range(K):
            e = int(idx[t, k])
            row = int(base[e // (E // P)]) + int(buf.slot_row[t, k])
            last = max(last, row)
            np.testing.assert_array_equal(buf.fp4.q[row].cpu().numpy(), ref.nibbles(codes)[0])
            want = wv[e] @ xv
            tol = H * 2.0 ** -23 * (np.abs(wv[e]) @ np.abs(xv))
            assert (np.abs(_f64(y[row]) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
    assert last * (H // 2) > 2 ** 32


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_gradient(layout):
    torch, dev = _dev()
    P, E, S, K, H = 8, 8, 50_000, 8, 7168  # 400000 rows, 5.7 GB each of y and dy
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    idx = torch.rand((S, E), generator=g, device=dev).argsort(1).to(torch.int32).contiguous()
    wts = torch.rand((S, K), generator=g, device=dev)
    dout = _normal(torch, dev, S, H, 6)
    y = _normal(torch, dev, S * K, H, 7)
    dy = torch.zeros_like(y)
    dw = torch.zeros((S, K), dtype=torch.float32, device=dev)
    err = torch.zeros(4, dtype=torch.int32, device=dev)
    base = torch.arange(P + 1, device=dev) * S  # every token goes to every rank: row g of each
    token = torch.arange(S, dtype=torch.int32, device=dev)[:, None].expand(S, K).contiguous()
    call = moe.moe_combine_expert_grad if layout == "expert" else moe.moe_combine_grad
    call(moe.make_shape(P, E, S, K, H), dout, y, 2 * H, base, S * K, token, idx, wts, dy, 2 * H, dw, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    for t in _some(S, 30):
        d32 = bf16_bits_to_f32(dout[t].cpu().numpy().view(np.uint16))
        for k in range(K):
            row = int(idx[t, k]) * S + int(t)
            want = f32_to_bf16_bits_torch(np.float32(wts[t, k].item()) * d32)
            np.testing.assert_array_equal(dy[row].cpu().numpy().view(np.uint16), want)
            terms = d32.astype(np.float64) * _f64(y[row])
            assert abs(float(dw[t, k]) - terms.sum()) <= H * 2.0 ** -24 * np.abs(terms).sum()
