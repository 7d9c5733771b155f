"""Combine's gradient on the GPU, both layouts. dy is one binary32 product rounded to bf16: bit for
bit. dw is a binary32 sum of H exact products: within H * 2^-24 * sum |dout y| of the 64-bit sum,
whatever the order. Differences: out is linear in y and in the weights, so the loss sum(dout * out),
taken in 64 bits at two points, has the gradient as its slope up to dw's and dy's own rounding."""

import numpy as np
import pytest

import oracle
from combine_moe_layout_02_gb300 import inputs, moe
from tests import gpu_path as gp
from tests.helpers import bf16_bits_to_f32, f32_to_bf16_bits_torch

pytestmark = pytest.mark.gpu


def _tables(w, layout):
    """(part base, send_head or slot_row) of the oracle."""
    _, nt = gp.oracle_tables(w)
    if layout == "rank":
        return nt["part_row_base"], nt["send_head"]
    ex = oracle.notify_expert(w.P, w.E, w.topk_idx, nt["num_recv_tokens_per_expert"], nt["recv_expert_offset"])
    return ex["expert_part_base"], ex["slot_row"]


def _routes(w, layout, base, routes):
    """Per token the (row, weights' slots) that combine reads, in its order."""
    epr = w.E // w.P
    out = []
    for g in range(w.S):
        rows = []
        if layout == "expert":
            for k in range(w.K):
                e = w.topk_idx[g, k]
                if 0 <= e < w.E:
                    rows.append((int(base[e // epr] + routes[g, k]), [k]))
        else:
            for d in range(w.P):
                if routes[g, d] >= 0:
                    rows.append((int(base[d] + routes[g, d]),
                                 [k for k in range(w.K) if 0 <= w.topk_idx[g, k] < w.E and w.topk_idx[g, k] // epr == d]))
        out.append(rows)
    return out


def _run(w, layout, weights=True, want_dy=True, want_dw=True, pad=0, seed=0):
    import torch

    dev = torch.device("cuda", 0)
    base, routes = _tables(w, layout)
    total = max(1, int(base[-1]))
    rng = np.random.default_rng(seed)
    dout = f32_to_bf16_bits_torch(rng.standard_normal((w.S, w.H)))
    y = np.full((total, w.H + pad), 0x7FC0, np.uint16)
    y[:, :w.H] = f32_to_bf16_bits_torch(rng.standard_normal((total, w.H)))
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    shape = moe.make_shape(w.P, w.E, w.S, w.K, w.H, w.C, w.expert_alignment)
    dy = torch.full((total, w.H + pad), 0x5555, dtype=torch.int16, device=dev) if want_dy else None
    dw = torch.full((w.S, w.K), -7.0, dtype=torch.float32, device=dev) if want_dw else None
    err = torch.zeros(4, dtype=torch.int32, device=dev)
    call = moe.moe_combine_expert_grad if layout == "expert" else moe.moe_combine_grad
    call(shape, up(dout.view(np.int16)), up(y.view(np.int16)) if want_dw else None, 2 * (w.H + pad), up(base), total,
         up(routes), up(w.topk_idx), up(w.topk_weights) if weights else None, dy, 2 * (w.H + pad), dw, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    d32, y64 = bf16_bits_to_f32(dout), bf16_bits_to_f32(y[:, :w.H]).astype(np.float64)
    want = np.full((total, w.H + pad), 0x5555, np.uint16)
    dots, tol = np.zeros((w.S, w.K)), np.zeros((w.S, w.K))
    for g, rows in enumerate(_routes(w, layout, base, routes)):
        for row, slots in rows:
            c = np.float32(0.0)
            for k in slots:
                c = np.float32(c + w.topk_weights[g, k])
            if layout == "expert":
                c = w.topk_weights[g, slots[0]]
            if not weights:
                c = np.float32(1.0)
            want[row, :w.H] = f32_to_bf16_bits_torch(c * d32[g])
            terms = d32[g].astype(np.float64) * y64[row]
            dots[g, slots], tol[g, slots] = terms.sum(), w.H * 2.0 ** -24 * np.abs(terms).sum()
    if want_dy:
        np.testing.assert_array_equal(dy.cpu().numpy().view(np.uint16), want)
    if want_dw:
        got = dw.cpu().numpy().astype(np.float64)
        assert (np.abs(got - dots) <= tol).all(), np.abs(got - dots).max()
    return dict(base=base, routes=routes, dout=d32, y=y64, dy=dy, dw=dw)


SHAPES = [(4, 16, 64, 256, 2, 0.0), (1, 8, 40, 72, 3, 0.2), (5, 5, 33, 8, 5, 0.4), (8, 64, 50, 264, 6, 0.15),
          (128, 256, 3, 7168, 8, 0.1), (1024, 1024, 1, 64, 16, 0.0), (16, 64, 100, 1032, 16, 0.6), (8, 32, 1, 4096, 1, 0.0)]


@pytest.mark.parametrize("layout", ["expert", "rank"])
@pytest.mark.parametrize("P,E,T,H,K,mask", SHAPES)
def test_gradient(layout, P, E, T, H, K, mask):
    w = inputs.make(P, E, T, H, K, seed=P + H, mask_frac=mask)
    if mask >= 0.4:
        w.topk_idx[::3] = -1  # tokens that reach no expert
    _run(w, layout)


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_many_tokens_take_a_warp_each(layout):
    _run(inputs.make(4, 16, 400, 136, 3, seed=4, mask_frac=0.1), layout)


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_without_weights_and_one_output_at_a_time(layout):
    w = inputs.make(8, 32, 40, 200, 4, seed=2, mask_frac=0.2, expert_alignment=16)
    _run(w, layout, weights=False)
    _run(w, layout, want_dw=False)
    _run(w, layout, want_dy=False)
    _run(w, layout, pad=8)


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_an_expert_twice_in_a_token(layout):
    w = inputs.make(4, 8, 30, 64, 4, seed=6)
    w.topk_idx[:, 2] = w.topk_idx[:, 0]
    w.topk_idx[::5] = 3
    _run(w, layout)


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_differences(layout):
    w = inputs.make(4, 8, 12, 40, 3, seed=8, mask_frac=0.2)
    r = _run(w, layout)
    routes = _routes(w, layout, r["base"], r["routes"])
    wt = w.topk_weights.astype(np.float64)

    def loss(y, c):
        return sum(float((r["dout"][g].astype(np.float64) * y[row]).sum()) * c[g, slots].sum()
                   for g, rows in enumerate(routes) for row, slots in rows)

    rng = np.random.default_rng(1)
    dw = r["dw"].cpu().numpy().astype(np.float64)
    dy = bf16_bits_to_f32(r["dy"].cpu().numpy().view(np.uint16)).astype(np.float64)
    h = 2.0 ** -6
    for _ in range(20):
        g, k = rng.integers(0, w.S), rng.integers(0, w.K)
        up, down = wt.copy(), wt.copy()
        up[g, k] += h
        down[g, k] -= h
        slope = (loss(r["y"], up) - loss(r["y"], down)) / (2 * h)
        mag = np.abs(r["dout"][g]).sum() * np.abs(r["y"]).max()
        assert abs(slope - dw[g, k]) <= w.H * 2.0 ** -24 * mag + 1e-9
    rows = [row for rows in routes for row, _ in rows]
    for _ in range(20):
        row, col = rng.choice(rows), rng.integers(0, w.H)
        up, down = r["y"].copy(), r["y"].copy()
        up[row, col] += h
        down[row, col] -= h
        slope = (loss(up, wt) - loss(down, wt)) / (2 * h)
        # one binary32 product of a weight that is a binary32 sum of up to K, rounded to bf16
        assert abs(slope - dy[row, col]) <= (2.0 ** -8 + 2.0 ** -22) * abs(slope) + 1e-9


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_rows_past_the_arena_are_skipped(layout):
    import torch

    w = inputs.make(2, 8, 20, 64, 3, seed=3)
    dev = torch.device("cuda", 0)
    base, routes = _tables(w, layout)
    keep = int(base[-1]) - 7
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    dout = up(f32_to_bf16_bits_torch(np.ones((w.S, w.H))).view(np.int16))
    y = torch.zeros((int(base[-1]), w.H), dtype=torch.int16, device=dev)
    dy = torch.full_like(y, 0x5555)
    dw = torch.full((w.S, w.K), -7.0, dtype=torch.float32, device=dev)
    err = torch.zeros(4, dtype=torch.int32, device=dev)
    call = moe.moe_combine_expert_grad if layout == "expert" else moe.moe_combine_grad
    shape = moe.make_shape(w.P, w.E, w.S, w.K, w.H)
    call(shape, dout, y, 2 * w.H, up(base), keep, up(routes), up(w.topk_idx), up(w.topk_weights), dy, 2 * w.H, dw, err)
    torch.cuda.synchronize()
    assert int(err[0]) == moe.MOE_ERR_CAPACITY
    assert (dy[keep:] == 0x5555).all() and not (dy[:keep] == 0x5555).all(dim=1).any()
    assert (dw == 0).all()


def test_dispatch_gradient_is_the_unweighted_combine():
    """dx of dispatch is the sum of its rows' gradients: combine without weights."""
    import torch

    w = inputs.make(4, 16, 24, 128, 3, seed=5, mask_frac=0.2)
    dev = torch.device("cuda", 0)
    base, routes = _tables(w, "expert")
    rng = np.random.default_rng(0)
    grad = f32_to_bf16_bits_torch(rng.standard_normal((int(base[-1]), w.H)))
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    dx = torch.empty((w.S, w.H), dtype=torch.int16, device=dev)
    err = torch.zeros(4, dtype=torch.int32, device=dev)
    moe.moe_combine_expert(moe.make_shape(w.P, w.E, w.S, w.K, w.H), up(grad.view(np.int16)), 2 * w.H, up(base), int(base[-1]),
                           up(routes), up(w.topk_idx), None, dx, err)
    got = bf16_bits_to_f32(dx.cpu().numpy().view(np.uint16)).astype(np.float64)
    g64 = bf16_bits_to_f32(grad).astype(np.float64)
    want = np.zeros((w.S, w.H))
    mag = np.zeros((w.S, w.H))
    for g, rows in enumerate(_routes(w, "expert", base, routes)):
        for row, _ in rows:
            want[g] += g64[row]
            mag[g] += np.abs(g64[row])
    assert (np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + mag * 2.0 ** -22) + w.K * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("layout", ["expert", "rank"])
def test_ids_that_name_no_expert_and_rows_that_are_nobodys(layout):
    """Ids past the experts give weights' gradients of 0 and no row; NaN in rows of the arena that no slot has reaches nothing."""
    import torch

    w = inputs.make(4, 8, 20, 64, 3, seed=11, mask_frac=0.1, expert_alignment=8)
    base, routes = _tables(w, layout)
    dev = torch.device("cuda", 0)
    idx = w.topk_idx.copy()
    idx[2, 1], idx[7, 0] = w.E, 2 ** 31 - 1
    total = int(base[-1])
    kept = w.topk_idx
    w.topk_idx = idx  # the tables are those of the valid ids; these two slots now name no expert
    rows = _routes(w, layout, base, routes)
    if layout == "rank":  # a rank's row stays with the slots that still name it
        rows = [[(row, slots) for row, slots in r if slots] for r in rows]
    used = {row for r in rows for row, _ in r}
    rng = np.random.default_rng(2)
    y = f32_to_bf16_bits_torch(rng.standard_normal((total, w.H)))
    y[[r for r in range(total) if r not in used]] = 0x7FC0
    dout = f32_to_bf16_bits_torch(rng.standard_normal((w.S, w.H)))
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    dy = torch.full((total, w.H), 0x5555, dtype=torch.int16, device=dev)
    dw = torch.full((w.S, w.K), -7.0, dtype=torch.float32, device=dev)
    err = torch.zeros(4, dtype=torch.int32, device=dev)
    call = moe.moe_combine_expert_grad if layout == "expert" else moe.moe_combine_grad
    call(moe.make_shape(w.P, w.E, w.S, w.K, w.H, expert_alignment=8), up(dout.view(np.int16)), up(y.view(np.int16)), 2 * w.H,
         up(base), total, up(routes), up(idx), up(w.topk_weights), dy, 2 * w.H, dw, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    got = dy.cpu().numpy().view(np.uint16)
    for r in range(total):
        assert (got[r] == 0x5555).all() == (r not in used), r
    g = dw.cpu().numpy()
    assert np.isfinite(g).all() and g[2, 1] == 0 and g[7, 0] == 0 and (g[kept < 0] == 0).all()
    d64, y64 = bf16_bits_to_f32(dout).astype(np.float64), bf16_bits_to_f32(y).astype(np.float64)
    for t, r in enumerate(rows):
        for row, slots in r:
            terms = d64[t] * y64[row]
            assert (np.abs(g[t, slots] - terms.sum()) <= w.H * 2.0 ** -24 * np.abs(terms).sum()).all()
