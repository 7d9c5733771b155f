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


def _tiled_rows(sf, rows, at, width):
    """Scale codes [len(at), width / 32] of rows `at` of an operand, on the host."""
    import torch

    chunks = -(-width // 128)
    part = sf.view(-1, chunks, 512)[torch.from_numpy(at // 128).to(sf.device)].cpu().numpy()
    words = np.stack([part[i, :, m % 32 * 16 + m % 128 // 32 * 4:][:, :4].reshape(-1) for i, m in enumerate(at)])
    return words[:, :width // 32]


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("N,K", [(1056, 4128), (1024, 4384)])
def test_product_in_clusters_of_two_pairs(gated, N, K):
    """Enough work on rows whose codes are no multiple of 128 bytes; an odd number of weight tiles and an even one."""
    torch, dev = _dev()
    counts = [3000, 2900, 0, 5001, 2500, 3100, 257, 3500]
    E, first, total = len(counts), [], 0
    for n in counts:
        first.append(total)
        total += -(-n // 128) * 128
    g = torch.Generator(device=dev)
    g.manual_seed(N)
    draw = lambda shape, lo, hi: torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.uint8)
    wt, ch = -(-N // 128), -(-K // 128)
    xq, wq = draw((total, K // 2), 0, 256), draw((E * N, K // 2), 0, 256)
    xsf, wsf = draw((total // 128, ch, 512), 125, 128), draw((E * wt, ch, 512), 120, 123)
    past = K % 128 // 32  # scales past the width are 0
    for sf in (xsf, wsf):
        sf.view(-1, ch, 128, 4)[:, -1, :, past:] = 0
    shape = moe.make_shape(1, E, sum(counts), 1, K, expert_alignment=128)
    plan, err = moe.expert_plan_buffer(shape, dev), torch.zeros(4, dtype=torch.int32, device=dev)
    moe.moe_expert_plan(shape, torch.tensor([counts], dtype=torch.int32, device=dev), plan, err)
    back = N // 2 if gated else N
    y = torch.full((total, back), 0x5555, dtype=torch.int16, device=dev)
    moe.moe_expert_product_fp4(E, N, K, gated, wq, wsf, xq, xsf, total, plan, y, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    wv = ref.values(ref.unnibble(wq.cpu().numpy()), np.concatenate(
        [ref.untiled(p, N, K) for p in wsf.view(E, -1).cpu().numpy()])).reshape(E, N, K)
    mine = np.zeros(total, bool)
    for e, (f, n) in enumerate(zip(first, counts)):
        mine[f:f + n] = True
        if n == 0:
            continue
        at = np.unique(np.concatenate([[f, f + n - 1, f + n // 2], f + np.arange(0, n, 211)]))
        xv = ref.values(ref.unnibble(xq[torch.from_numpy(at).to(dev)].cpu().numpy()), _tiled_rows(xsf, total, at, K))
        v, m = xv @ wv[e].T, K * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv[e]).T)
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
    gap = torch.from_numpy(np.flatnonzero(~mine)).to(dev)
    assert (y[gap] == 0x5555).all()


def test_expert_layer_in_clusters_of_two_pairs():
    """The packing epilogue there: the bits of the operators one after another."""
    torch, dev = _dev()
    E, S, K, H, inner = 8, 4300, 4, 4128, 544
    shape = moe.make_shape(1, E, S, K, H, expert_alignment=128)
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
    buf.expert_ffn_fp4(*args, two, h=h)  # bf16 inner rows, packed by a launch of their own
    torch.cuda.synchronize()
    assert int(buf.err[0]) == 0
    assert torch.equal(one, two)
