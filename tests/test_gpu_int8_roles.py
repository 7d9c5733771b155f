"""Every role of the int8 product's forms gives up on its own: the converting warps of each group, and the last warp that takes
sums out, in tiles of 64, 128 and 256 rows and with K shared by pairs."""

import time

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests.test_gpu_int8_product import _err, _operands, _plan, _up

pytestmark = pytest.mark.gpu

FORMS = {
    # E, N, K, rows of the experts
    "256 rows": (6, 4192, 1040, [300, 1, 0, 700, 129, 400]),
    "128 rows": (68, 1056, 1040, [31] * 60 + [130, 256, 257, 700, 0, 1, 128, 129]),
    "64 rows": (64, 1056, 1040, [2] * 60 + [0, 70, 1, 3]),
    "shared K": (1, 512, 4112, [300]),
}


@pytest.mark.parametrize("quit_warp", [3, 4, 7, 8, 9, 10, 11])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_warp_of_every_kind_gives_up(form, quit_warp):
    import torch

    E, N, K, counts = FORMS[form]
    counts = np.array(counts)
    plan, first = _plan(E, counts) if E > 1 else (None, [0, counts[0]])
    rows = int(first[-1])
    operands = _up(*_operands(E, N, K, rows, 1))
    err = _err()
    y = [torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    call = lambda out: moe.moe_expert_product_int8(E, N, K, 0, *operands, rows, plan, out, err)
    call(y[0])
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    moe.moe_test_product_wait(20_000_000, quit_warp)  # about 10 ms
    began = time.perf_counter()
    call(y[1])
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 10.0
    assert int(err[0]) == moe.MOE_ERR_DEVICE_TIMEOUT
    err.zero_()
    call(y[2])  # the hook armed one call only
    torch.cuda.synchronize()
    assert int(err[0]) == 0 and torch.equal(y[0], y[2])


@pytest.mark.parametrize("rows,fit", [(100, 1), (129, 2), (200, 2), (257, 3), (300, 3)])
def test_a_plan_of_more_rows_than_there_are_is_reported(rows, fit):
    """Tiles behind the rows are skipped and reported, however many there are; the others are computed."""
    import torch

    E, N, K = 5, 64, 64
    plan, first = _plan(E, np.full(E, 1))
    a, b, c, d = _up(*_operands(E, N, K, rows, 2))
    got = []
    for n in (rows, int(first[-1])):
        x, s = torch.zeros((n, K), dtype=torch.int8, device="cuda"), torch.zeros((n,), device="cuda")
        x[:rows], s[:rows] = c, d
        y, err = torch.full((n, N), 7.0, dtype=torch.bfloat16, device="cuda"), _err()
        moe.moe_expert_product_int8(E, N, K, 0, a, b, x, s, n, plan, y, err)
        got.append((y, int(err[0])))
    assert got[0][1] == moe.MOE_ERR_CAPACITY and got[1][1] == 0
    live = torch.arange(rows, device="cuda") % 128 == 0
    assert int(live.sum()) == fit and (got[0][0][live] != 7).any(1).all()
    assert torch.equal(got[0][0], got[1][0][:rows])
