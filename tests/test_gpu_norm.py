"""The norm, its gradient and int8 rows on the GPU against 64 bits."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import router_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = 2.0 ** -24       # half a step of binary32
BF = 2.0 ** -8       # half a step of bf16


def _bf16(shape, seed, scale=1.0):
    import torch

    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def _np(t):
    return t.detach().double().cpu().numpy()


def _rel(H):
    """Relative error of rstd and what is multiplied by it: a sum of H squares by threads of at most 32 values, 5 steps of a
    warp and 31 warps (half a unit each, halved by the root), a quotient, a sum, a root, two products."""
    return (34 + 5 + 31 + 8) * U


WIDTHS = [8, 16, 24, 256, 264, 1000, 1024, 1040, 2048, 2056, 4096, 7168, 8200, 16384]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5])
def test_norm(H, rows):
    import torch

    x, r, w = _bf16((rows, H), 1), _bf16((rows, H), 2, 4.0), _bf16((H,), 3)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    for residual in (True, False):
        h = _np(x) + (_np(r) if residual else 0)
        v, _ = ref.rms(h, _np(w), EPS)
        y, s = torch.empty_like(xd), torch.empty_like(xd)
        moe.moe_rms_norm(xd, wd, EPS, y=y, residual=rd if residual else None, sum_out=s)
        assert (np.abs(_np(s) - h) <= np.abs(h) * (BF + U)).all()
        assert (np.abs(_np(y) - v) <= np.abs(v) * (BF + _rel(H) * (1 + BF))).all()
        if H % 16 == 0:
            q = torch.empty((rows, H), dtype=torch.int8, device="cuda")
            qs = torch.empty((rows,), device="cuda")
            moe.moe_rms_norm(xd, wd, EPS, residual=rd if residual else None, q=q, q_scale=qs)
            scale = np.abs(v).max(1) / 127
            assert (np.abs(_np(qs) - scale) <= scale * (_rel(H) + 2 * U)).all()
            # v / scale is off by 127 times their relative errors, and the code by half
            off = np.abs(_np(q) - v / scale[:, None])
            assert (off <= 0.5 + 127 * (2 * _rel(H) + 4 * U)).all() and np.abs(_np(q)).max() == 127
            # all results at once are the same bits, in place where that is allowed
            y2, q2, qs2, r2, x2 = torch.empty_like(xd), torch.empty_like(q), torch.empty_like(qs), rd.clone(), xd.clone()
            moe.moe_rms_norm(x2, wd, EPS, y=x2, residual=r2 if residual else None, sum_out=r2 if residual else None, q=q2,
                             q_scale=qs2)
            assert torch.equal(x2, y) and torch.equal(q2, q) and torch.equal(qs2, qs)
            assert not residual or torch.equal(r2, s)


@pytest.mark.parametrize("H", [16, 272, 7168])
def test_rows_apart(H):
    """Every array's rows at a distance of its own; what lies between stays. int8 rows in dispatch's slots."""
    import torch

    rows = 37
    wide = lambda pad, seed: _bf16((rows, H + pad), seed).cuda()
    x, r, w = wide(8, 1), wide(24, 2), _bf16((H,), 3).cuda()
    y, s = torch.full((rows, H + 16), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows, H + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    stride = moe.moe_slot_stride(H, 1)
    at = (H + 31) // 32 * 32
    arena = torch.full((rows, stride), 7, dtype=torch.int8, device="cuda")
    scales = arena[:, at:at + 4].view(torch.float32)
    moe.moe_rms_norm(x[:, :H], w, EPS, y=y[:, :H], residual=r[:, :H], sum_out=s[:, :H], q=arena[:, :H], q_scale=scales)
    want = [torch.empty((rows, H), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, qs = torch.empty((rows, H), dtype=torch.int8, device="cuda"), torch.empty((rows,), device="cuda")
    moe.moe_rms_norm(x[:, :H].contiguous(), w, EPS, y=want[0], residual=r[:, :H].contiguous(), sum_out=want[1], q=q, q_scale=qs)
    assert torch.equal(y[:, :H], want[0]) and torch.equal(s[:, :H], want[1])
    assert torch.equal(arena[:, :H], q) and torch.equal(scales[:, 0], qs)
    assert (y[:, H:] == 7).all() and (s[:, H:] == 7).all() and (arena[:, H:at] == 7).all() and (arena[:, at + 4:] == 7).all()


@pytest.mark.parametrize("H", [16, 1024, 7168])
def test_rows_of_zeros_infinities_and_far_values(H):
    import torch

    x = _bf16((9, H), 1)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] *= 2.0 ** 100   # squares past binary32
    x[4] = torch.finfo(torch.bfloat16).max
    x[5] *= 2.0 ** -60   # eps is far above the squares
    x[6, 0] = 2.0 ** 90
    w = _bf16((H,), 2)
    y, q = torch.empty_like(x).cuda(), torch.empty((9, H), dtype=torch.int8, device="cuda")
    qs = torch.empty((9,), device="cuda")
    moe.moe_rms_norm(x.cuda(), w.cuda(), EPS, y=y, q=q, q_scale=qs)
    fine = [0, 3, 4, 5, 6, 7, 8]
    v, _ = ref.rms(_np(x)[fine], _np(w), EPS)
    assert (np.abs(_np(y)[fine] - v) <= np.abs(v) * (BF + _rel(H) * (1 + BF)) + 1e-40).all()
    assert not q[0].any() and qs[0] == 0 and qs[1:3].isnan().all() and not q[1:3].any() and qs[fine].isfinite().all()
    scale = np.abs(v).max(1, keepdims=True) / 127
    near = np.abs(_np(q)[fine][1:] - (v / np.where(scale > 0, scale, 1))[1:])
    assert (near <= 0.5 + 127 * (2 * _rel(H) + 4 * U)).all()
    # the gradient at the same rows
    dy, dh = _bf16((9, H), 4), torch.empty_like(y)
    moe.moe_rms_norm_grad(dy.cuda(), x.cuda(), w.cuda(), EPS, dh)
    want, _, mag, _ = ref.rms_grad(_np(dy)[fine], _np(x)[fine], _np(w), EPS)
    # binary32 holds the gradient's factors of the rows of 2^100 as numbers of fewer bits: rstd^2 h^2 in two steps
    assert (np.abs(_np(dh)[fine] - want) <= np.abs(want) * BF + mag * (2 * _rel(H) + 80 * U) + 1e-37).all()


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_gradient(H, rows):
    import torch

    dy, h, w, ds = _bf16((rows, H), 1), _bf16((rows, H), 2, 3.0), _bf16((H,), 3), _bf16((rows, H), 4)
    for dsum in (None, ds):
        dh, dw = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda"), torch.empty((H,), device="cuda")
        scratch = moe.rms_norm_grad_scratch(rows, H)
        scratch.fill_(255)
        moe.moe_rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), EPS, dh, dweight=dw, dsum=None if dsum is None else dsum.cuda(),
                              scratch=scratch)
        want, wdw, mag, wmag = ref.rms_grad(_np(dy), _np(h), _np(w), EPS, None if dsum is None else _np(dsum))
        assert (np.abs(_np(dh) - want) <= np.abs(want) * BF + mag * (2 * _rel(H) + 80 * U) * (1 + BF)).all()
        # a block's rows and the blocks, half a unit each, and every term's own
        assert (np.abs(_np(dw) - wdw) <= wmag * (_rel(H) + (min(rows, 608) + rows / 152 + 4) * U)).all()
        only = torch.empty_like(dh)
        moe.moe_rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), EPS, only, dsum=None if dsum is None else dsum.cuda())
        assert torch.equal(only, dh)


def test_gradient_in_place_apart_and_without_rows():
    import torch

    rows, H = 65, 1040
    wide = lambda pad, seed: _bf16((rows, H + pad), seed).cuda()
    dy, h, ds, w = wide(8, 1), wide(16, 2), wide(24, 3), _bf16((H,), 4).cuda()
    want = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_rms_norm_grad(dy[:, :H].contiguous(), h[:, :H].contiguous(), w, EPS, want, dsum=ds[:, :H].contiguous())
    tail = ds[:, H:].clone()
    moe.moe_rms_norm_grad(dy[:, :H], h[:, :H], w, EPS, ds[:, :H], dsum=ds[:, :H])
    assert torch.equal(ds[:, :H], want) and torch.equal(ds[:, H:], tail)
    dw = torch.full((H,), 7.0, device="cuda")
    none = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_rms_norm_grad(none, none, w, EPS, none, dweight=dw, scratch=moe.rms_norm_grad_scratch(0, H))
    assert not dw.any()
    moe.moe_rms_norm(none, w, EPS, y=none)


@pytest.mark.parametrize("rows,width", [(1, 16), (3, 48), (40, 256), (17, 1040), (5, 7168), (2, 16400), (3, 32768)])
def test_int8_rows_are_exact(rows, width):
    import torch

    x = _bf16((rows, width), width)
    x[0, :16] = torch.tensor([127.0, 0.5, 1.5, -2.5, 63.5, 126.5, -0.5, 3.25] * 2)  # ties, where 127 is the largest
    x[0, 16:] *= 8
    x[0].clamp_(-127, 127)
    if rows > 2:
        x[1] = 0
        x[2] *= 2.0 ** -120
    if rows > 4:
        x[3, 7] = float("nan")
        x[4, 2] = -float("inf")
    if rows > 16:
        x[5] = torch.finfo(torch.bfloat16).max
        x[6] = 2.0 ** -133  # the smallest there is
        x[7] *= 2.0 ** -126
    op = moe.Int8Rows(rows, width).pack(x.cuda())
    q, s = ref.int8_rows(x.float().numpy())
    assert np.array_equal(op.q.cpu().numpy(), q)
    assert np.array_equal(op.scale.cpu().numpy().view(np.uint32)[~np.isnan(s)], s.view(np.uint32)[~np.isnan(s)])
    assert np.array_equal(op.scale.isnan().cpu().numpy(), np.isnan(s))
    back = op.unpack(torch.empty_like(x).cuda())
    want = torch.from_numpy(q.astype(np.float32) * s[:, None]).to(torch.bfloat16)
    assert torch.equal(back.cpu().nan_to_num(9.0), want.nan_to_num(9.0))


def test_int8_rows_are_dispatch_s():
    """The same bits as the int8 dispatch writes into its slots."""
    import torch

    from combine_moe_layout_02_gb300 import inputs

    w = inputs.make(1, 8, 300, 2064, 1, seed=5)
    shape = moe.make_shape(1, 8, 300, 1, 2064, quant=1)
    buf = moe.Buffers(shape, "cuda")
    x = torch.from_numpy(w.x_bits.view(np.int16)).cuda().view(torch.bfloat16)
    idx = torch.from_numpy(w.topk_idx).cuda()
    buf.layout(idx)
    buf.notify()
    buf.dispatch(x, idx, torch.from_numpy(w.topk_weights).cuda())
    op = moe.Int8Rows(300, 2064).pack(x)
    rows = buf.recv_arena.view(torch.int8)[buf.send_head[:, 0].long()]
    assert torch.equal(rows[:, :2064], op.q)
    at = (2064 + 31) // 32 * 32
    assert torch.equal(rows[:, at:at + 4].contiguous().view(torch.float32)[:, 0], op.scale)


def test_gated_rows():
    import torch

    groups, rows, width = 3, 96, 80
    x = _bf16((groups * rows, width), 1)
    op = moe.Int8Rows(rows, width, groups=groups, gated=True).pack(x.cuda())
    src = np.concatenate([g * rows + ref.gated_order(rows) for g in range(groups)])
    q, s = ref.int8_rows(x.float().numpy()[src])
    assert np.array_equal(op.q.cpu().numpy(), q) and np.array_equal(op.scale.cpu().numpy(), s)
    back = op.unpack(torch.empty_like(x).cuda()).float().cpu().numpy()
    want = torch.from_numpy(q.astype(np.float32) * s[:, None]).to(torch.bfloat16).float().numpy()
    assert np.array_equal(back[src], want)


def test_a_plan_s_rows_only():
    import torch

    E, K, S, width = 5, 2, 400, 272
    counts = np.array([[0, 1, 300, 129, 370]], np.int32)
    shape = moe.make_shape(1, E, S, K, 64, expert_alignment=128)
    plan = moe.expert_plan_buffer(shape)
    moe.moe_expert_plan(shape, torch.from_numpy(counts).cuda(), plan)
    first = np.concatenate([[0], np.cumsum((counts[0] + 127) // 128 * 128)])
    rows = int(first[-1]) + 50
    x = _bf16((rows, width), 1)
    op = moe.Int8Rows(rows, width)
    op.q.fill_(7), op.scale.fill_(7)
    op.pack(x.cuda(), E=E, plan=plan)
    mine = np.zeros(rows, bool)
    for e in range(E):
        mine[first[e]:first[e] + counts[0, e]] = True
    q, s = ref.int8_rows(x.float().numpy())
    got, gs = op.q.cpu().numpy(), op.scale.cpu().numpy()
    assert np.array_equal(got[mine], q[mine]) and np.array_equal(gs[mine], s[mine])
    assert (got[~mine] == 7).all() and (gs[~mine] == 7).all()
    out = torch.full_like(x, 7.0).cuda()
    op.unpack(out, E=E, plan=plan)
    want = torch.from_numpy(q.astype(np.float32) * s[:, None]).to(torch.bfloat16).float().numpy()
    o = out.float().cpu().numpy()
    assert np.array_equal(o[mine], want[mine]) and (o[~mine] == 7).all()


def test_in_a_graph_and_on_another_stream():
    import torch

    rows, H = 333, 2048
    w = _bf16((H,), 9).cuda()
    inputs = [[_bf16((rows, H), 10 * i + j).cuda() for j in range(4)] for i in range(2)]

    def step(x, r, dy, ds, out):
        moe.moe_rms_norm(x, w, EPS, residual=r, sum_out=out["sum"], y=out["y"], q=out["op"].q, q_scale=out["op"].scale)
        moe.moe_rms_norm_grad(dy, out["sum"], w, EPS, out["dh"], dweight=out["dw"], dsum=ds, scratch=out["scratch"])
        out["op"].unpack(out["back"])

    def fresh():
        e = lambda: torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
        return dict(sum=e(), y=e(), dh=e(), back=e(), dw=torch.empty((H,), device="cuda"), op=moe.Int8Rows(rows, H),
                    scratch=moe.rms_norm_grad_scratch(rows, H))

    names = ("sum", "y", "dh", "back", "dw")
    want = []
    for a in inputs:
        o = fresh()
        step(*a, o)
        want.append([o[n].clone() for n in names])
    held = [t.clone() for t in inputs[0]]
    o = fresh()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*held, o)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(*held, o)
    for i in (1, 0, 1):
        for a, b in zip(held, inputs[i]):
            a.copy_(b)
        o["scratch"].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for n, b in zip(names, want[i]):
            assert torch.equal(o[n], b), n


@pytest.mark.parametrize("H", [7168])
def test_past_32_bits_of_offset(H):
    """Rows whose byte offsets pass 2^32."""
    import torch

    rows = (1 << 32) // (2 * H) + 300
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    tail = _bf16((128, H), 1).cuda()
    x[-128:] = tail
    w = _bf16((H,), 2).cuda()
    y, q, qs = torch.empty_like(x), torch.empty((rows, H), dtype=torch.int8, device="cuda"), torch.empty((rows,), device="cuda")
    moe.moe_rms_norm(x, w, EPS, y=y, q=q, q_scale=qs)
    a, b, c = torch.empty_like(tail), torch.empty((128, H), dtype=torch.int8, device="cuda"), torch.empty((128,), device="cuda")
    moe.moe_rms_norm(tail, w, EPS, y=a, q=b, q_scale=c)
    assert torch.equal(y[-128:], a) and torch.equal(q[-128:], b) and torch.equal(qs[-128:], c) and not y[:-128].any()
    dh, g = torch.empty_like(x), torch.empty_like(tail)
    moe.moe_rms_norm_grad(x, x, w, EPS, dh)
    moe.moe_rms_norm_grad(tail, tail, w, EPS, g)
    assert torch.equal(dh[-128:], g)


@pytest.mark.parametrize("power", [-100, -84, -83, -82, -40, 0, 60, 120])
def test_int8_rows_of_every_bf16_quotient(power):
    """Each largest value of a power of two with each value down to 2^-9 of it: quotients at and beside ties."""
    import torch

    mantissas = np.arange(128, 256, dtype=np.float32)
    below = np.concatenate([mantissas * np.float32(2.0) ** -k for k in range(10)])
    rows = []
    for m in mantissas:
        v = np.where(below <= m, below, np.float32(0))
        rows.append(np.concatenate([[m], v, -v, np.zeros(15)]).astype(np.float32))
    x = (np.stack(rows) * np.float32(2.0) ** (power - 7)).astype(np.float32)
    xd = torch.from_numpy(x).to(torch.bfloat16)
    assert (xd.float().numpy() == x).all()
    scale = np.abs(x).max(1) / np.float32(127)
    want = np.rint(x / scale[:, None])
    op = moe.Int8Rows(*x.shape).pack(xd.cuda())
    assert np.array_equal(op.q.cpu().numpy(), want.astype(np.int8)) and np.array_equal(op.scale.cpu().numpy(), scale)
