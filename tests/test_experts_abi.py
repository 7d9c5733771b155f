"""The experts' operators answer bad arguments on the host (no GPU; the fake pointers are never read)."""

import pytest

from combine_moe_layout_02_gb300 import build as moe_build
from combine_moe_layout_02_gb300 import moe
from tests import fp4_ref as ref

A = 1 << 20  # an aligned address
BAD, UNSUP = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def test_sizes(lib):
    assert moe.moe_fp4_scale_bytes(0, 32) == 0
    assert moe.moe_fp4_scale_bytes(1, 32) == 512
    assert moe.moe_fp4_scale_bytes(129, 160) == 2 * 2 * 512
    assert moe.moe_fp4_scale_bytes(128, 7168) == 56 * 512
    assert moe.moe_fp4_scale_bytes(-1, 32) == -1 and moe.moe_fp4_scale_bytes(1, 48) == -1
    s = moe.make_shape(8, 256, 64, 8, 7168, expert_alignment=128)
    assert moe.moe_expert_plan_ints(s) == 4 + 2 * 256 + 4 * (256 + 2)
    assert moe.moe_expert_plan_ints(moe.make_shape(8, 256, 64, 8, 7168, expert_alignment=64)) == -1
    assert moe.moe_expert_plan_ints(moe.make_shape(8, 250, 64, 8, 7168, expert_alignment=128)) == -1


@pytest.mark.parametrize("name", ["moe_fp4_pack", "moe_fp4_unpack"])
def test_pack_refusals(lib, name):
    def call(groups=1, rows=128, width=64, gated=0, x=A, stride=128, q=A, sf=A, E=0, plan=None, ints=0):
        # both take (.., x or q, ..); the checks do not depend on which is read
        if name == "moe_fp4_pack":
            return lib.moe_fp4_pack(groups, rows, width, gated, x, stride, q, sf, E, plan, ints, None)
        return lib.moe_fp4_unpack(groups, rows, width, gated, q, sf, x, stride, E, plan, ints, None)

    assert call(groups=-1) == BAD and call(rows=-1) == BAD
    assert call(width=0) == BAD and call(width=48) == BAD and call(width=32800, stride=1 << 20) == UNSUP
    assert call(gated=2) == BAD and call(gated=1, rows=48) == BAD
    assert call(stride=127) == BAD and call(stride=112) == BAD and call(stride=136) == BAD
    assert call(x=None) == BAD and call(q=None) == BAD and call(sf=None) == BAD
    assert call(x=A + 8) == BAD and call(q=A + 4) == BAD and call(sf=A + 1) == BAD
    assert call(groups=1 << 30, rows=1 << 30) == UNSUP
    ints = 4 + 2 * 8
    assert call(E=8, plan=A, ints=ints - 1) == BAD and call(E=0, plan=A, ints=ints) == BAD
    assert call(E=8, plan=A + 4, ints=ints) == BAD and call(E=8, plan=A, ints=ints, rows=64) == BAD
    assert call(E=8, plan=A, ints=ints, groups=2) == BAD and call(E=8, plan=A, ints=ints, gated=1) == BAD
    assert call(rows=0, x=None, q=None, sf=None) == moe.MOE_OK  # nothing to do


def test_plan_and_dispatch_refusals(lib):
    s = moe.make_shape(4, 16, 64, 2, 64, expert_alignment=128)
    n = moe.moe_expert_plan_ints(s)
    assert lib.moe_expert_plan(s, A, A, n - 1, None, None) == BAD
    assert lib.moe_expert_plan(s, None, A, n, None, None) == BAD
    assert lib.moe_expert_plan(s, A, None, n, None, None) == BAD
    assert lib.moe_expert_plan(s, A, A, n, A + 2, None) == BAD
    assert lib.moe_expert_plan(moe.make_shape(4, 16, 64, 2, 64), A, A, n, None, None) == BAD
    args = lambda **k: {**dict(x=A, i=A, w=None, r=A, b=A, q=A, sf=A, rows=128), **k}

    def call(shape=s, **k):
        a = args(**k)
        return lib.moe_dispatch_expert_fp4(shape, a["x"], a["i"], a["w"], a["r"], a["b"], a["q"], a["sf"], a["rows"], None,
                                           None, None, None)

    for name in ("x", "i", "r", "b", "q", "sf"):
        assert call(**{name: None}) == BAD and call(**{name: A + 8}) == BAD, name
    assert call(rows=-1) == BAD
    assert call(shape=moe.make_shape(4, 16, 64, 2, 72, expert_alignment=128)) == BAD  # H not a multiple of 32


def test_product_refusals(lib):
    def call(E=2, N=64, K=64, gated=0, wq=A, wsf=A, xq=A, xsf=A, rows=128, plan=A, ints=64, y=A, stride=128, err=None):
        return lib.moe_expert_product_fp4(E, N, K, gated, wq, wsf, xq, xsf, rows, plan, ints, y, stride, err, None)

    assert call(E=0) == BAD and call(N=0) == BAD and call(K=0) == BAD
    assert call(N=48, stride=96) == BAD and call(K=48) == BAD and call(gated=2) == BAD
    assert call(E=4097, ints=1 << 20) == UNSUP and call(K=32800) == UNSUP and call(N=65568, stride=1 << 20) == UNSUP
    assert call(rows=-128) == BAD and call(rows=100) == BAD and call(rows=1 << 31) == UNSUP
    assert call(stride=126) == BAD and call(stride=120) == BAD and call(gated=1, stride=48) == BAD
    for name in ("wq", "wsf", "xq", "xsf", "plan", "y"):
        assert call(**{name: None}) == BAD and call(**{name: A + 8}) == BAD, name
    assert call(err=A + 1) == BAD and call(ints=7) == BAD
    assert call(rows=0, xq=None, xsf=None, y=None) == moe.MOE_OK


def test_ffn_refusals(lib):
    s = moe.make_shape(4, 16, 64, 2, 64, expert_alignment=128)
    need = moe.moe_expert_ffn_fp4_workspace_bytes(s, 96)
    assert need > 0 and moe.moe_expert_ffn_fp4_rows(s, 96) == 128 * 17
    assert moe.moe_expert_ffn_fp4_workspace_bytes(s, 48) == -1
    assert moe.moe_expert_ffn_fp4_workspace_bytes(moe.make_shape(4, 16, 64, 2, 72), 96) == -1

    def call(shape=s, inner=96, x=A, i=A, w=A, a=A, b=A, c=A, d=A, h=None, out=A, ws=A, n=need, err=None):
        return lib.moe_expert_ffn_fp4(shape, inner, x, i, w, a, b, c, d, h, out, ws, n, err, None)

    for name in ("x", "i", "a", "b", "c", "d", "out", "ws"):
        assert call(**{name: None}) == BAD and call(**{name: A + 8}) == BAD, name
    for name in ("w", "h"):
        assert call(**{name: A + 8}) == BAD, name
    assert call(n=need - 1) == BAD and call(ws=A + 16) == BAD and call(err=A + 1) == BAD
    assert call(inner=0) == BAD and call(inner=32800) == UNSUP
    assert call(shape=moe.make_shape(4, 16, 64, 2, 72)) == BAD
    empty = moe.make_shape(4, 16, 0, 2, 64)
    assert call(shape=empty, x=None, i=None, out=None, n=moe.moe_expert_ffn_fp4_workspace_bytes(empty, 96)) == moe.MOE_OK


@pytest.mark.parametrize("name", ["moe_combine_grad", "moe_combine_expert_grad"])
def test_gradient_refusals(lib, name):
    s = moe.make_shape(4, 16, 64, 2, 64)

    def call(shape=s, dout=A, y=A, ys=128, base=A, rows=64, routes=A, i=A, w=A, dy=A, dys=128, dw=A, err=None):
        return getattr(lib, name)(shape, dout, y, ys, base, rows, routes, i, w, dy, dys, dw, err, None)

    for arg in ("dout", "y", "base", "routes", "i"):
        assert call(**{arg: None}) == BAD and call(**{arg: A + 8}) == BAD, arg
    assert call(dy=None, dw=None) == BAD
    assert call(dy=A + 8) == BAD and call(dw=A + 4) == BAD and call(w=A + 4) == BAD and call(err=A + 2) == BAD
    assert call(ys=112) == BAD and call(ys=136) == BAD and call(dys=112) == BAD and call(dys=136) == BAD
    assert call(rows=-1) == BAD and call(shape=moe.make_shape(4, 15, 64, 2, 64)) == BAD


def test_reference_rounds_as_the_format_says():
    """The 64-bit reference itself, at values worked out by hand."""
    import numpy as np

    x = np.zeros((1, 32))
    x[0, :8] = [8.0, 7.0, 5.0, 5.01, 0.5, 0.51, -3.0, 1.0]  # largest 8: scale 2, grid 0, 1, 2, 3, 4, 6, 8, 12
    codes, s = ref.pack(x)
    assert s[0, 0] == 127 + 1
    assert list(codes[0, :8]) == [6, 6, 4, 5, 0, 1, 8 + 3, 1]
    v = ref.values(codes, s)[0, :8]
    assert list(v) == [8.0, 8.0, 4.0, 6.0, 0.0, 1.0, -3.0, 1.0]
