"""Calls whose results would overwrite what they still read are answered on the host (no GPU; the fake pointers are never read)."""

import pytest

from combine_moe_layout_02_gb300 import build as moe_build
from combine_moe_layout_02_gb300 import moe

A, B, C, D, E = (k << 20 for k in range(1, 6))  # aligned addresses, never read
BAD, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_OK


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def test_norm_in_place(lib):
    def call(x=A, xs=128, r=B, rs=128, o=C, os=128, y=D, ys=128, q=E, qs=64, rows=4):
        return lib.moe_rms_norm(rows, 64, 1e-6, x, xs, r, rs, 6 << 20, o, os, y, ys, q, qs, 7 << 20, 4, None)

    # the same rows at another distance
    assert call(o=A, os=144) == BAD and call(o=B, os=144) == BAD and call(y=A, ys=144) == BAD and call(y=B, ys=144) == BAD
    # int8 rows over any of the others
    for name in "ABCD":
        assert call(q=globals()[name]) == BAD, name
    assert call(rows=0, o=A, os=144) == OK


def test_norm_gradient_in_place(lib):
    def call(dy=A, dys=128, h=B, ds=C, dss=128, dh=D, dhs=128, rows=4):
        return lib.moe_rms_norm_grad(rows, 64, 1e-6, dy, dys, h, 128, 6 << 20, ds, dss, dh, dhs, None, None, 0, None)

    assert call(dh=A, dhs=144) == BAD and call(dh=C, dhs=144) == BAD and call(dh=B) == BAD
    assert call(rows=0, dh=B) == OK


@pytest.mark.parametrize("name", ["moe_int8_pack", "moe_int8_unpack"])
def test_int8_rows_in_place(lib, name):
    assert getattr(lib, name)(1, 4, 64, 0, A, 128, A, 128, B, 4, 0, None, 0, None) == BAD
