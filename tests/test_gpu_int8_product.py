"""The product of int8 operands on the GPU against 64 bits."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import inputs, moe
from tests import router_ref as ref

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


def _operands(E, N, K, rows, seed, big=False):
    """Random codes and scales; big: of few, large values, so that sums pass 2^24."""
    rng = np.random.default_rng(seed)
    draw = (lambda shape: rng.choice(np.array([127, -127, 126, 127, 127], np.int8), shape)) if big else (
        lambda shape: np.clip(np.rint(rng.normal(size=shape) * 32), -127, 127).astype(np.int8))
    scale = lambda shape, mid: (mid * (0.5 + rng.random(shape))).astype(np.float32)
    return (draw((E, N, K)), scale((E, N), 1 / 32 / np.sqrt(K)), draw((rows, K)), scale((rows,), 1 / 32))


def _up(*arrays):
    import torch

    return [torch.from_numpy(a).cuda() for a in arrays]


def _check(got, y, off, where=""):
    bad = np.abs(got - y) > np.abs(y) * BF + off * (1 + BF) + 1e-38
    assert not bad.any(), (where, np.argwhere(bad)[:4], got[bad][:4], y[bad][:4])


def _err():
    import torch

    return torch.zeros((4,), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("rows,N,K", [(1, 32, 16), (1, 4096, 7168), (2, 96, 48), (3, 64, 1040), (8, 160, 512), (9, 288, 64),
                                      (16, 64, 2048), (17, 512, 144), (31, 32, 32), (33, 256, 400), (100, 640, 272),
                                      (128, 64, 128), (129, 96, 4112), (255, 224, 208), (256, 256, 256), (257, 544, 176),
                                      (1000, 320, 96)])
def test_dense(rows, N, K, gated):
    import torch

    wq, ws, xq, xs = _operands(1, N, K, rows, rows + N + K)
    width = N // 2 if gated else N
    y = torch.full((rows + 1, width), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    a, b, c, d = _up(wq, ws, xq, xs)
    moe.moe_expert_product_int8(1, N, K, gated, a, b, c, d, rows, None, y, err)
    want, off = ref.product(wq[0], ws[0], xq, xs, gated)
    _check(y[:rows].double().cpu().numpy(), want, off)
    assert (y[rows:] == 7).all() and not err.any()


@pytest.mark.parametrize("rows", [1, 5, 40, 200])
def test_sums_past_24_bits(rows):
    import torch

    N, K = 64, 32768
    wq, ws, xq, xs = _operands(1, N, K, rows, rows, big=True)
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    a, b, c, d = _up(wq, ws, xq, xs)
    moe.moe_expert_product_int8(1, N, K, 0, a, b, c, d, rows, None, y, None)
    want, off = ref.product(wq[0], ws[0], xq, xs, False)
    _check(y.double().cpu().numpy(), want, off)


def test_whole_sums_are_exact():
    """Below 2^24 the sum is exact: with scales of 1 and results that bf16 holds nothing is off."""
    import torch

    rng = np.random.default_rng(1)
    for rows in (4, 70):
        K = 4096
        wq = rng.choice(np.array([-127, -3, 0, 1, 2, 127], np.int8), (64, K))
        xq = rng.choice(np.array([-127, -1, 0, 1, 5, 127], np.int8), (rows, K))
        acc = xq.astype(np.int64) @ wq.astype(np.int64).T
        assert np.abs(xq.astype(np.int64)).dot(np.abs(wq.astype(np.int64)).T).max() < 2 ** 25
        y = torch.empty((rows, 64), dtype=torch.bfloat16, device="cuda")
        a, b, c, d = _up(wq[None], np.ones((1, 64), np.float32), xq, np.ones(rows, np.float32))
        moe.moe_expert_product_int8(1, 64, K, 0, a, b, c, d, rows, None, y, None)
        assert torch.equal(y.cpu(), torch.from_numpy(acc.astype(np.float64)).to(torch.bfloat16))


def _plan(E, counts, K=8):
    import torch

    total = int(counts.sum())
    shape = moe.make_shape(1, E, max(-(-total // K), 1), K, 64, expert_alignment=128)
    plan = moe.expert_plan_buffer(shape)
    moe.moe_expert_plan(shape, torch.from_numpy(counts[None].astype(np.int32)).cuda(), plan)
    first = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    return plan, first


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("N,K,counts,slots", [
    (64, 32, [1], False), (96, 80, [0, 0, 3], False), (320, 256, [1, 0, 2, 300, 0, 31, 33, 128, 129, 5], True),
    (256, 1040, [600, 1, 1], True), (512, 144, [0, 256, 257, 255, 0, 64], False), (32, 16, [0, 0], False),
    (1056, 400, [2] * 40, True)])
def test_experts(N, K, counts, slots, gated):
    import torch

    counts = np.array(counts)
    E = len(counts)
    plan, first = _plan(E, counts)
    rows = int(first[-1]) + 3
    wq, ws, xq, xs = _operands(E, N, K, rows, N + K)
    mine = np.zeros(rows, bool)
    for e in range(E):
        mine[first[e]:first[e] + counts[e]] = True
    xs[~mine] = np.nan  # nobody's rows are nobody's business
    width = N // 2 if gated else N
    y = torch.full((rows, width + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    a, b, c, d = _up(wq, ws, xq, xs)
    kw = dict(y_row_stride=2 * (width + 8))
    if slots:
        stride, at = moe.moe_slot_stride(K, 1), (K + 31) // 32 * 32
        arena = torch.full((rows, stride), 7, dtype=torch.int8, device="cuda")
        arena[:, :K] = c
        arena[:, at:at + 4] = d.view(torch.int8).view(rows, 4)
        moe.moe_expert_product_int8(E, N, K, gated, a, b, arena, arena.data_ptr() + at, rows, plan, y, err,
                                    x_row_stride=stride, xs_stride=stride, **kw)
    else:
        moe.moe_expert_product_int8(E, N, K, gated, a, b, c, d, rows, plan, y, err, **kw)
    got = y.double().cpu().numpy()
    for e in range(E):
        at = slice(first[e], first[e] + counts[e])
        want, off = ref.product(wq[e], ws[e], xq[at], xs[at], gated)
        _check(got[at, :width], want, off, e)
    assert (got[~mine] == 7).all() and (got[:, width:] == 7).all() and not err.any()


def test_a_row_without_a_number():
    import torch

    wq, ws, xq, xs = _operands(1, 64, 64, 40, 1)
    for rows in (6, 40):
        s = xs.copy()
        s[3] = np.nan
        y = torch.empty((rows, 64), dtype=torch.bfloat16, device="cuda")
        a, b, c, d = _up(wq, ws, xq, s)
        moe.moe_expert_product_int8(1, 64, 64, 0, a, b, c, d, rows, None, y, None)
        assert y[3].isnan().all() and y[:3].isfinite().all() and y[4:].isfinite().all()


def test_plans_that_are_none():
    """Tiles outside the rows or of no expert are skipped and reported; the others are computed."""
    import torch

    E, N, K = 3, 64, 64
    counts = np.array([40, 128, 5])
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    wq, ws, xq, xs = _operands(E, N, K, rows, 2)
    a, b, c, d = _up(wq, ws, xq, xs)
    tiles = 4 + 2 * 4
    for field, value in ((0, 3), (0, -1), (1, rows - 64), (1, -128), (2, 257), (2, -1)):
        bad = plan.clone()
        bad[tiles + 4 * 1 + field] = value  # the second tile
        y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        err = _err()
        moe.moe_expert_product_int8(E, N, K, 0, a, b, c, d, rows, bad, y, err)
        assert err[0].item() == moe.MOE_ERR_CAPACITY, (field, value)
        for e in (0, 2):
            at = slice(first[e], first[e] + counts[e])
            want, off = ref.product(wq[e], ws[e], xq[at], xs[at], False)
            _check(y[at].double().cpu().numpy(), want, off)
        assert (y[first[1]:first[1] + counts[1]] == 7).all()
    many = plan.clone()
    many[0] = 1 << 30  # more tiles than the plan has room for
    none = plan.clone()
    none[0] = -5
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_product_int8(E, N, K, 0, a, b, c, d, rows, none, y, None)
    assert (y == 7).all()


def test_the_int8_expert_layer_end_to_end():
    """norm -> gate -> int8 dispatch -> gate and up -> pack -> down -> combine, in a graph, against 64 bits of each step."""
    import torch

    S, E, K, H, inner = 96, 8, 2, 512, 256
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(1)
    bf = lambda shape, s: torch.from_numpy((rng.normal(size=shape) * s).astype(np.float32)).to(torch.bfloat16).to(dev)
    x, r, w = bf((S, H), 1), bf((S, H), 2), bf((H,), 1)
    gate_up = moe.Int8Rows(2 * inner, H, dev, groups=E, gated=True).pack(bf((E * 2 * inner, H), H ** -0.5))
    down = moe.Int8Rows(H, inner, dev, groups=E).pack(bf((E * H, inner), inner ** -0.5))
    router = bf((E, H), H ** -0.5)
    shape = moe.make_shape(4, E, S, K, H, expert_alignment=128, quant=1)
    buf, gate = moe.Buffers(shape, dev, side_arrays=False), moe.Gate(shape, dev, balance=0.01)
    rows = moe.moe_max_expert_rows(shape)
    h, y = torch.zeros((S, H), dtype=torch.bfloat16, device=dev), torch.zeros((S, H), dtype=torch.bfloat16, device=dev)
    mid = torch.zeros((rows, inner), dtype=torch.bfloat16, device=dev)
    packed = moe.Int8Rows(rows, inner, dev)
    back = torch.zeros((rows, H), dtype=torch.bfloat16, device=dev)
    out = torch.zeros_like(x)
    logits = torch.zeros((S, E), dtype=torch.float32, device=dev)

    def step():
        moe.moe_rms_norm(x, w, 1e-6, y=y, residual=r, sum_out=h)
        torch.mm(y.float(), router.float().t(), out=logits)
        idx, weights = gate.forward(logits)
        buf.layout(idx)
        buf.notify()
        buf.notify_expert(idx)
        buf.expert_plan()
        buf.dispatch_expert(y, idx, weights)
        buf.expert_product_int8(gate_up, mid)
        packed.pack(mid, E=E, plan=buf.plan)
        moe.moe_expert_product_int8(E, H, inner, 0, down.q, down.scale, packed.q, packed.scale, rows, buf.plan, back, buf.err)
        buf.combine_expert(out, idx, weights, y=back, y_row_stride=2 * H)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(bf((S, H), 1))
    graph.replay()
    torch.cuda.synchronize()
    assert not buf.err.any()
    # every step against its definition on what the step before it gave
    to64 = lambda t: t.double().cpu().numpy()
    v, _ = ref.rms(to64(x) + to64(r), to64(w), 1e-6)
    assert (np.abs(to64(y) - v) <= np.abs(v) * (BF + 1e-5)).all()
    f = ref.gate(to64(logits), K, balance=0.01)
    assert np.array_equal(gate.topk_idx.cpu().numpy(), f["idx"])
    assert np.array_equal(buf.num_tokens_per_expert.sum(0).cpu().numpy(), f["count"][:E])
    yq, ys = ref.int8_rows(y.float().cpu().numpy())
    row = (buf.expert_part_base.cpu().numpy()[f["idx"] // (E // 4)] + buf.slot_row.cpu().numpy())
    gu, gus = gate_up.q.view(E, 2 * inner, H).cpu().numpy(), gate_up.scale.view(E, -1).cpu().numpy()
    dq, dqs = down.q.view(E, H, inner).cpu().numpy(), down.scale.view(E, -1).cpu().numpy()
    got = to64(mid)
    mq, msc = ref.int8_rows(mid.float().cpu().numpy())
    want_out = np.zeros((S, H))
    size = np.zeros((S, H))
    for g in range(S):
        for k in range(K):
            e, at = f["idx"][g, k], row[g, k]
            want, off = ref.product(gu[e], gus[e], yq[g:g + 1], ys[g:g + 1], True)
            _check(got[at:at + 1], want, off, (g, k))
            want, off = ref.product(dq[e], dqs[e], mq[at:at + 1], msc[at:at + 1], False)
            _check(to64(back)[at:at + 1], want, off, (g, k))
            term = float(gate.topk_weights[g, k]) * to64(back)[at]
            want_out[g] += term
            size[g] += np.abs(term)
    assert (np.abs(to64(out) - want_out) <= np.abs(want_out) * BF + size * 4 * ref.ULP).all()


def test_on_another_stream_and_the_same_bits_again():
    import torch

    E, N, K = 4, 256, 528
    counts = np.array([100, 0, 300, 7])
    plan, first = _plan(E, counts)
    rows = int(first[-1])
    a, b, c, d = _up(*_operands(E, N, K, rows, 3))
    want = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_product_int8(E, N, K, 0, a, b, c, d, rows, plan, want, None)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(side, outs):
            moe.moe_expert_product_int8(E, N, K, 0, a, b, c, d, rows, plan, o, None, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
