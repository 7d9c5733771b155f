"""Counts that no routing of the shape has: reported, and the plan names no row or tile beyond its own list."""

import pytest

from combine_moe_layout_02_gb300 import moe

pytestmark = pytest.mark.gpu


def _plan(P, E, S, K, counts):
    """(err, plan, the words past its end) for counts [P, E]."""
    import torch

    dev = torch.device("cuda", 0)
    shape = moe.make_shape(P, E, S, K, 64, expert_alignment=128)
    n = moe.moe_expert_plan_ints(shape)
    room = torch.full((n + 4096,), -7, dtype=torch.int32, device=dev)
    err = torch.zeros(4, dtype=torch.int32, device=dev)
    moe.moe_expert_plan(shape, counts.to(dev), room[:n], err)
    torch.cuda.synchronize()
    return int(err[0]), room[:n].cpu().numpy(), room[n:].cpu().numpy()


@pytest.mark.parametrize("P", [1, 4, 64])
def test_more_rows_than_a_routing_needs(P):
    """Each expert's count is possible, their rows together are not: no expert gets any."""
    import torch

    S, K, E = 128, 2, 64
    counts = torch.zeros((P, E), dtype=torch.int32)
    counts[P - 1, :2] = 128  # 256 = S * K: a routing's
    err, plan, past = _plan(P, E, S, K, counts)
    assert err == moe.MOE_OK and list(plan[:4]) == [2, 256, E, 0]
    counts[0, :] = 129  # 64 * 256 rows; a routing needs 256 + 64 * 127 at most
    counts[P - 1, :2] = 127
    err, plan, past = _plan(P, E, S, K, counts)
    assert err == moe.MOE_ERR_INCONSISTENT and list(plan[:4]) == [0, 0, E, 0]
    assert not plan[4:4 + 2 * E].any() and (plan[4 + 2 * E:] == -7).all() and (past == -7).all()


@pytest.mark.parametrize("P,count", [(1, 1 << 28), (4, 1 << 26), (64, 1 << 22)])
def test_counts_whose_tiles_pass_32_bits(P, count):
    """4096 experts with every slot each: 2^32 tiles."""
    import torch

    err, plan, past = _plan(P, 4096, 1 << 24, 16, torch.full((P, 4096), count, dtype=torch.int32))
    assert err == moe.MOE_ERR_INCONSISTENT
    assert plan[0] == 0 and plan[1] == 0 and not plan[4:4 + 2 * 4096].any()
    assert (plan[4 + 2 * 4096:] == -7).all() and (past == -7).all()  # no tile was listed
