"""The gate's gradient where a program has dropped the slots near the row's largest logit: what is left lies far below it."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import router_ref as ref
from tests.test_gpu_gate import HALF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("E", [6, 12, 30, 60, 100, 256, 700, 1300])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_slots_far_below_the_dropped_ones(E, dtype, scale):
    """D is the sum over the slots that are left: their shares of it, and so the gradient, do not depend on how far down they are."""
    import torch

    depths = [20.0, 60.0, 80.0, 84.0, 85.5, 86.0, 86.5, 87.0, 87.5, 90.0, 104.0, 200.0, 600.0]
    S, K = len(depths) * 4, 5
    rng = np.random.default_rng(E)
    z = rng.normal(size=(S, E))
    for i, depth in enumerate(depths):  # two dropped slots up there, three kept ones that far below
        rows = slice(4 * i, 4 * i + 4)
        z[rows, 2:5] += 6 - depth
        z[rows, 5:] -= 6 + depth
    zt = torch.from_numpy(z).to(getattr(torch, dtype))
    z64 = zt.double().numpy()
    f = ref.gate(z64, K, None, True, scale, 0.1)
    idx = f["idx"].copy()
    assert (np.sort(idx[:, :2]) == [0, 1]).all() and (np.sort(idx[:, 2:]) == [2, 3, 4]).all()
    idx[:, :2] = -1
    idx[1::4, 2] = idx[1::4, 3]  # one id twice
    idx[2::4, 4] = -1
    op = moe.Gate(moe.make_shape(1, E, S, K, 64), "cuda", normalize=True, scale=scale, balance=0.1)
    op.forward(zt.cuda())
    op.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    dw = rng.normal(size=(S, K)).astype(np.float32)
    got = op.backward(zt.cuda(), torch.from_numpy(dw).cuda(), torch.ones(1, device="cuda")).double().cpu().numpy()
    want, mag = ref.gate_grad(f, idx, dw, 1.0, True, scale, 0.1)
    # as test_gpu_gate's bound; a probability below 2^-126 is 0, and meets numbers (c - T) below 1
    tol = mag * (4 * ref.gate_rel(z64) + (E / 32 + 30) * ref.ULP) + np.abs(want) * HALF[dtype] + 2.0 ** -126
    assert (np.abs(f["prob"]) <= 1).all() and np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), np.argwhere(np.abs(got - want) > tol)[:4]
    # what is left decides: three slots of ordinary weights give gradients of their size
    assert (np.abs(want[::4, 2:5]).max(1) > 1e-3).all()


def test_nothing_left_that_counts():
    """Slots with ids of experts at -infinity alone, or none: no gradient of the weights, and no NaN."""
    import torch

    for E in (10, 200, 1200):
        z = torch.zeros((3, E))
        z[:, 4:] = -float("inf")
        op = moe.Gate(moe.make_shape(1, E, 3, 2, 64), "cuda", normalize=True)
        op.forward(z.cuda())
        op.topk_idx.copy_(torch.tensor([[5, 6], [-1, -1], [E, 7]], dtype=torch.int32))
        assert not op.backward(z.cuda(), torch.ones((3, 2), device="cuda")).any()
