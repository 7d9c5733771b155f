"""The gate and its gradient on the GPU against 64 bits."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import router_ref as ref

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}


def _logits(S, E, dtype, seed, banned=0.0, spread=1.5):
    import torch

    g = torch.Generator().manual_seed(seed)
    z = torch.randn((S, E), generator=g) * spread
    z[torch.rand((S, E), generator=g) < banned] = -float("inf")
    return z.to(getattr(torch, dtype))


def _gate(S, E, K, **kw):
    return moe.Gate(moe.make_shape(1, E, S, K, 64), "cuda", **kw)


def _check_forward(op, f, z, scale):
    rel = ref.gate_rel(z)
    got = {n: getattr(op, n).cpu().numpy() for n in ("topk_idx", "topk_weights", "expert_count", "expert_prob", "loss")}
    assert np.array_equal(got["topk_idx"], f["idx"])
    assert np.array_equal(got["expert_count"], f["count"])
    # a weight: two probabilities' errors, their sum's 16 additions, a quotient and a product
    w = f["weights"]
    assert (np.abs(got["topk_weights"] - w) <= np.abs(w) * (2 * rel + 12 * ref.ULP)).all()
    # a mean: positive terms, each sum of a warp, a block and the call rounds: at most one rounding per token
    steps = min(len(z), 512) + 640
    assert (np.abs(got["expert_prob"] - f["prob"]) <= f["prob"] * (rel + steps * ref.ULP / 2)).all()
    tol = np.abs(f["loss"]) * (rel + (steps + z.shape[1] / 32 + 40) * ref.ULP / 2)
    assert abs(float(got["loss"][0]) - f["loss"]) <= tol + 1e-45


def _check_backward(got, f, z, idx, dw, dloss, normalize, scale, balance, dtype):
    want, mag = ref.gate_grad(f, idx, dw, dloss, normalize, scale, balance)
    # each term is a product of at most four probabilities' worth of error; sums of E and K terms
    tol = mag * (4 * ref.gate_rel(z) + (z.shape[1] / 32 + 30) * ref.ULP) + np.abs(want) * HALF[dtype] + 1e-40
    assert (np.abs(got.float().cpu().numpy() - want) <= tol).all()


CASES = [
    # S, E, K, dtype, normalize, scale, balance, banned, masked
    (1, 256, 8, "float32", True, 1.0, 0.01, 0.0, 0.0),
    (1, 1, 1, "float32", False, 1.0, 0.5, 0.0, 0.0),
    (7, 5, 5, "bfloat16", True, 2.5, 1.0, 0.0, 0.0),
    (33, 3, 8, "float32", True, 1.0, 0.01, 0.0, 0.3),      # fewer experts than slots
    (64, 16, 2, "bfloat16", False, 1.0, 0.01, 0.0, 0.0),
    (257, 31, 4, "float32", False, 16.0, 0.1, 0.5, 0.2),
    (129, 33, 16, "bfloat16", True, 1.0, 0.01, 0.9, 0.5),  # most rows end before the slots do
    (300, 64, 6, "bfloat16", True, 1.0, 0.01, 0.0, 0.0),
    (1000, 250, 6, "bfloat16", False, 1.0, 0.01, 0.3, 0.1),
    (515, 256, 8, "bfloat16", True, 1.0, 0.01, 0.0, 0.0),
    (401, 384, 8, "float32", True, 1.0, 0.01, 0.0, 0.0),
    (77, 513, 9, "bfloat16", True, 1.0, 0.01, 0.1, 0.0),
    (50, 1024, 16, "float32", True, 1.0, 0.01, 0.0, 0.0),
    (43, 1025, 7, "float32", False, 1.0, 0.01, 0.0, 0.1),
    (19, 4096, 16, "bfloat16", True, 1.0, 0.01, 0.0, 0.0),
]


@pytest.mark.parametrize("S,E,K,dtype,normalize,scale,balance,banned,masked", CASES)
def test_gate_and_gradient(S, E, K, dtype, normalize, scale, balance, banned, masked):
    import torch

    z = _logits(S, E, dtype, S + E, banned)
    rng = np.random.default_rng(S)
    mask = (rng.random(S) >= masked).astype(np.uint8) if masked else None
    op = _gate(S, E, K, normalize=normalize, scale=scale, balance=balance)
    zd = z.cuda()
    md = torch.from_numpy(mask).cuda() if mask is not None else None
    ids, weights = op.forward(zd, mask=md)
    torch.cuda.synchronize()
    assert ids is op.topk_idx and weights is op.topk_weights
    z64 = z.double().numpy()
    f = ref.gate(z64, K, mask, normalize, scale, balance)
    _check_forward(op, f, z64, scale)

    dw = rng.normal(size=(S, K)).astype(np.float32)
    dwd, dl = torch.from_numpy(dw).cuda(), torch.tensor([0.7], device="cuda")
    got = op.backward(zd, dwd, dl, mask=md)
    assert got.dtype == z.dtype
    dl64 = float(np.float32(0.7))
    _check_backward(got, f, z64, f["idx"], dw, dl64, normalize, scale, balance, dtype)
    # either gradient alone, into rows of the caller's
    only = torch.full_like(zd, 7.0)
    assert op.backward(zd, dwd, None, mask=md, dlogits=only) is only
    _check_backward(only, f, z64, f["idx"], dw, 0.0, normalize, scale, balance, dtype)
    _check_backward(op.backward(zd, None, dl, mask=md), f, z64, f["idx"], 0 * dw, dl64, normalize, scale, balance, dtype)
    assert not op.backward(zd, mask=md).float().any()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("E", [6, 40, 256, 700, 2000])
def test_rows_apart(E, dtype):
    """Logits and their gradient as columns of wider tensors, at odd distances; what lies between stays."""
    import torch

    S, K = 70, 4
    z = _logits(S, E + 3, dtype, E).cuda()
    op = _gate(S, E, K, balance=0.1)
    op.forward(z[:, :E])
    z64 = z[:, :E].double().cpu().numpy()
    f = ref.gate(z64, K, balance=0.1)
    _check_forward(op, f, z64, 1.0)
    dw = torch.randn((S, K), generator=torch.Generator().manual_seed(1)).cuda()
    out = torch.full((S, E + 5), 7.0, dtype=z.dtype, device="cuda")
    op.backward(z[:, :E], dw, torch.ones(1, device="cuda"), dlogits=out[:, :E])
    _check_backward(out[:, :E], f, z64, f["idx"], dw.cpu().numpy(), 1.0, True, 1.0, 0.1, dtype)
    assert (out[:, E:] == 7).all()


@pytest.mark.parametrize("E", [8, 200, 1500])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_ties_go_to_the_lowest_expert(E, dtype):
    import torch

    z = torch.zeros((5, E), dtype=getattr(torch, dtype))
    z[1, E // 2:] = 1
    z[2, ::2] = -0.0
    z[3] = torch.arange(E) % 2
    z[4, E - 1] = 2
    op = _gate(5, E, 4)
    op.forward(z.cuda())
    want = ref.gate(z.double().numpy(), 4)["idx"]
    assert want[2].tolist() == [0, 1, 2, 3]
    assert np.array_equal(op.topk_idx.cpu().numpy(), want)


@pytest.mark.parametrize("E", [6, 256, 1100])
def test_infinities_and_nan(E):
    import torch

    S, K = 8, 3
    z = _logits(S, E, "float32", 3)
    z[1] = -float("inf")
    z[2, 4] = float("nan")
    z[3, 5] = float("inf")
    z[4, 1:] = -float("inf")
    z[5] = torch.finfo(torch.float32).min  # the type's lowest value is a number
    z[6] = float("nan")
    op = _gate(S, E, K, balance=1.0)
    op.forward(z.cuda())
    got, w = op.topk_idx.cpu().numpy(), op.topk_weights.cpu().numpy()
    want = ref.gate(np.where(np.isinf(z.double().numpy()) & (z.double().numpy() > 0), 1e300, z.double().numpy()), K)["idx"]
    assert np.array_equal(got, want)
    assert got[1].tolist() == [-1] * 3 and got[4].tolist() == [0, -1, -1] and got[5].tolist() == [0, 1, 2]
    assert got[2][0] == 4 and got[3][0] == 5 and got[6].tolist() == [0, 1, 2]
    for g in (2, 3, 6):
        assert np.isnan(w[g]).all()
    for g in (0, 4, 5, 7):
        f = ref.gate(z[g:g + 1].double().numpy(), K)
        assert (np.abs(w[g] - f["weights"][0]) <= f["weights"][0] * (2 * ref.gate_rel(z[g:g + 1].double().numpy()) + 12 * ref.ULP)).all()
    assert not w[1].any() and np.isnan(op.loss.item())
    assert op.expert_count.cpu().numpy().sum() == (got >= 0).sum() + 7
    # no row's gradient reads another's: without the rows that hold none, the others' are the same bits
    dw = torch.randn((S, K), generator=torch.Generator().manual_seed(1)).cuda()
    dz = op.backward(z.cuda(), dw, torch.ones(1, device="cuda"))
    assert dz[[2, 3, 6]].isnan().any(1).all() and not dz[1].any() and dz[[0, 4, 5, 7]].isfinite().all()


@pytest.mark.parametrize("E", [50, 256, 1000, 1200])
def test_large_logits(E):
    """Logits whose neighbours in binary32 are as far apart as their exponentials: only differences count."""
    import torch

    g = torch.Generator().manual_seed(E)
    z = torch.randint(0, 16, (40, E), generator=g).float()
    z[:10] += 2.0 ** 23
    z[10:20] -= 2.0 ** 23
    z[20:30] = z[20:30] * 2.0 ** 100  # one or a few experts take all
    z[30:] = torch.where(z[30:] > 7, torch.finfo(torch.float32).max, torch.finfo(torch.float32).min)
    op = _gate(40, E, 6, balance=0.1)
    op.forward(z.cuda())
    z64 = z.double().numpy()
    f = ref.gate(z64, 6, balance=0.1)
    assert np.array_equal(op.topk_idx.cpu().numpy(), f["idx"])
    rel = ref.gate_rel(np.minimum(z64[:20] - z64[:20].min(1, keepdims=True), 16))
    w = f["weights"]
    assert (np.abs(op.topk_weights.cpu().numpy() - w) <= w * (2 * rel + 12 * ref.ULP)).all()
    dw = torch.randn((40, 6), generator=g)
    dz = op.backward(z.cuda(), dw.cuda(), torch.ones(1, device="cuda"))
    want, mag = ref.gate_grad(f, f["idx"], dw.double().numpy(), 1.0, True, 1.0, 0.1)
    tol = mag * (4 * rel + (E / 32 + 30) * ref.ULP) + np.abs(want) * 2.0 ** -24 + 1e-37
    assert (np.abs(dz.double().cpu().numpy() - want) <= tol).all()


def test_no_token_is_routed():
    import torch

    op = _gate(40, 16, 2, balance=1.0)
    z = _logits(40, 16, "float32", 1).cuda()
    for mask, zz in ((torch.zeros(40, dtype=torch.bool, device="cuda"), z), (None, torch.full_like(z, -float("inf")))):
        op.forward(zz, mask=mask)
        assert (op.topk_idx == -1).all() and not op.topk_weights.any() and not op.expert_count.any()
        assert not op.expert_prob.any() and op.loss.item() == 0
        assert not op.backward(zz, torch.ones((40, 2), device="cuda"), torch.ones(1, device="cuda"), mask=mask).any()


def test_no_tokens():
    import torch

    op = _gate(0, 16, 2, balance=1.0)
    op.forward(torch.empty((0, 16), device="cuda"))
    assert not op.expert_count.any() and not op.expert_prob.any() and op.loss.item() == 0
    assert op.backward(torch.empty((0, 16), device="cuda"), torch.empty((0, 2), device="cuda")).shape == (0, 16)


@pytest.mark.parametrize("E", [12, 256, 1300])
@pytest.mark.parametrize("normalize", [True, False])
def test_ids_that_a_program_changed(E, normalize):
    """Dropped slots, ids past the experts and the same id twice."""
    import torch

    S, K = 90, 5
    z = _logits(S, E, "float32", E)
    op = _gate(S, E, K, normalize=normalize, scale=1.5, balance=0.2)
    zd = z.cuda()
    op.forward(zd)
    z64 = z.double().numpy()
    f = ref.gate(z64, K, None, normalize, 1.5, 0.2)
    rng = np.random.default_rng(3)
    idx = f["idx"].copy()
    idx[rng.random((S, K)) < 0.3] = -1
    idx[rng.random((S, K)) < 0.1] = E
    idx[5] = -1
    idx[10:30, 1] = idx[10:30, 0]
    idx[20:40, 4] = idx[20:40, 0]
    op.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    dw = rng.normal(size=(S, K)).astype(np.float32)
    dz = op.backward(zd, torch.from_numpy(dw).cuda(), torch.ones(1, device="cuda"))
    _check_backward(dz, f, z64, idx, dw, 1.0, normalize, 1.5, 0.2, "float32")


@pytest.mark.parametrize("S,E", [(20000, 256), (3000, 1024)])
def test_many_tokens(S, E):
    import torch

    z = _logits(S, E, "bfloat16", S)
    op = _gate(S, E, 8, balance=0.01)
    zd = z.cuda()
    op.forward(zd)
    zz = zd.double()
    idx = torch.sort(zz, dim=1, descending=True, stable=True).indices[:, :8]
    assert torch.equal(op.topk_idx.long(), idx)
    p = torch.softmax(zz, 1)
    rel = ref.gate_rel(z[:64].double().numpy()) * 1.5
    w = p.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    assert ((op.topk_weights - w).abs() <= w * (2 * rel + 12 * ref.ULP)).all()
    assert ((op.expert_prob - p.mean(0)).abs() <= p.mean(0) * (rel + 1200 * ref.ULP / 2)).all()
    count = torch.bincount(idx.flatten(), minlength=E)
    assert torch.equal(op.expert_count[:E].long(), count) and op.expert_count[E].item() == S


def test_same_bits_again_in_a_graph_and_on_another_stream():
    import torch

    S, E, K = 3001, 250, 6
    z = [_logits(S, E, "bfloat16", i).cuda() for i in range(2)]
    dw, dl = torch.randn((S, K), device="cuda"), torch.ones(1, device="cuda")
    names = ("topk_idx", "topk_weights", "expert_count", "expert_prob", "loss")
    want = []
    for zz in z:
        op = _gate(S, E, K, balance=0.1)
        op.forward(zz)
        dz = op.backward(zz, dw, dl)
        want.append([getattr(op, n).clone() for n in names] + [dz])
    op = _gate(S, E, K, balance=0.1)
    x, dz = z[0].clone(), torch.empty_like(z[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        op.forward(x)
        op.backward(x, dw, dl, dlogits=dz)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        op.forward(x)
        op.backward(x, dw, dl, dlogits=dz)
    for i in (1, 0, 1):
        x.copy_(z[i])
        op.scratch.fill_(255)  # nothing is carried over
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([getattr(op, n) for n in names] + [dz], want[i]):
            assert torch.equal(a, b)
    # a stream given by its handle
    op.forward(z[0], stream=side.cuda_stream)
    out = op.backward(z[0], dw, dl, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0][5]) and torch.equal(op.loss, want[0][4])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("S,E,K,normalize,banned,masked", [
    (1, 8, 2, True, 0.0, 0.0),
    (31, 8, 16, True, 0.0, 0.3),      # twice as many slots as experts
    (2049, 8, 1, False, 0.2, 0.0),
    (15, 16, 16, True, 0.0, 0.0),     # all experts of all tokens
    (5000, 16, 2, True, 0.3, 0.1),
    (999, 24, 5, False, 0.5, 0.2),
    (8, 32, 4, True, 0.0, 1.0),       # no token is routed
    (3001, 60, 4, True, 0.0, 0.0),
    (70000, 64, 8, True, 0.1, 0.1),   # several turns of every warp
    (257, 65, 6, True, 0.0, 0.0),     # a warp to a token from here on
    (70000, 9, 3, False, 0.0, 0.5),
])
def test_tokens_that_share_a_warp(S, E, K, normalize, banned, masked, dtype):
    test_gate_and_gradient(S, E, K, dtype, normalize, 1.5, 0.05, banned, masked)


def test_buffers_elsewhere_are_refused():
    import torch

    op = moe.Gate(moe.make_shape(1, 8, 4, 2, 64), "cpu")
    z = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError, match="the gate's buffers are on cpu"):
        op.forward(z)
    with pytest.raises(ValueError, match="the gate's buffers are on cpu"):
        op.backward(z)
    op = _gate(4, 8, 2)
    with pytest.raises(ValueError):
        op.forward(torch.zeros((4, 8)))
    op.forward(z)
    with pytest.raises(moe.MoeError):
        op.backward(z, dlogits=z)
