"""The gate, the norm and the int8 operators answer bad arguments on the host (no GPU; the fake pointers are never read)."""

import pytest
import torch

from combine_moe_layout_02_gb300 import build as moe_build
from combine_moe_layout_02_gb300 import moe

A = 1 << 20  # an aligned address
BAD, UNSUP = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def test_gate_refusals(lib):
    s = moe.make_shape(1, 16, 64, 2, 64)
    need = lib.moe_gate_scratch_bytes(s)
    assert need > 0 and lib.moe_gate_scratch_bytes(moe.make_shape(1, 0, 64, 2, 64)) == -1

    def call(shape=s, kind=0, z=A, stride=64, mask=None, normalize=1, idx=A, w=A, c=A, p=A, loss=A, ws=A, n=need):
        return lib.moe_gate(shape, kind, z, stride, mask, normalize, 1.0, 0.0, idx, w, c, p, loss, ws, n, None)

    for name in ("z", "idx", "w", "c", "ws"):
        assert call(**{name: None}) == BAD and call(**{name: A + 8}) == BAD, name
    assert call(p=A + 8) == BAD and call(loss=A + 2) == BAD and call(ws=A + 16) == BAD and call(n=need - 1) == BAD
    assert call(kind=2) == BAD and call(kind=-1) == BAD and call(normalize=2) == BAD
    assert call(stride=60) == BAD and call(stride=66) == BAD and call(kind=1, stride=31) == BAD
    assert call(shape=moe.make_shape(1, 16, 64, 17, 64)) == UNSUP
    assert call(shape=moe.make_shape(1, 4097, 64, 2, 64), stride=1 << 20, n=1 << 40) == UNSUP


def test_gate_gradient_refusals(lib):
    s = moe.make_shape(1, 16, 64, 2, 64)

    def call(shape=s, kind=0, z=A, stride=64, normalize=1, idx=A, c=A, dw=A, dl=A, dz=A + 4096, dstride=64):
        return lib.moe_gate_grad(shape, kind, z, stride, None, normalize, 1.0, 0.0, idx, c, dw, dl, dz, dstride, None)

    for name in ("z", "idx", "c", "dz"):
        assert call(**{name: None}) == BAD and call(**{name: A + 8}) == BAD, name
    assert call(dw=A + 4) == BAD and call(dl=A + 1) == BAD
    assert call(kind=3) == BAD and call(normalize=-1) == BAD and call(stride=60) == BAD and call(dstride=60) == BAD
    assert call(dstride=65) == BAD
    assert call(dz=A) == BAD  # over the logits
    empty = moe.make_shape(1, 16, 0, 2, 64)
    assert call(shape=empty, z=None, idx=None, dz=None) == moe.MOE_OK


def test_norm_refusals(lib):
    def call(rows=4, H=64, eps=1e-6, x=A, xs=128, r=A, rs=128, w=A, o=A, os=128, y=A + 4096, ys=128, q=A, qs=64, s=A, ss=4):
        return lib.moe_rms_norm(rows, H, eps, x, xs, r, rs, w, o, os, y, ys, q, qs, s, ss, None)

    assert call(rows=-1) == BAD and call(H=0) == BAD and call(H=12) == BAD
    assert call(H=16392, xs=1 << 16, rs=1 << 16, os=1 << 16, ys=1 << 16, qs=1 << 16) == UNSUP
    assert call(H=72, xs=144, rs=144, os=144, ys=144, qs=80) == BAD  # int8 rows of 8 values
    for eps in (0.0, -1e-6, INF, NAN, 1e-39):
        assert call(eps=eps) == BAD, eps
    assert call(x=None) == BAD and call(w=None) == BAD
    for name in ("x", "r", "w", "o", "y", "q"):
        assert call(**{name: A + 8}) == BAD, name
    for name in ("xs", "rs", "os", "ys", "qs"):
        assert call(**{name: 8}) == BAD and call(**{name: 200}) == BAD, name
    assert call(s=None) == BAD and call(q=None) == BAD and call(s=A + 2) == BAD and call(ss=2) == BAD and call(ss=6) == BAD
    assert call(o=None, y=None, q=None, s=None) == BAD  # nothing asked for
    assert call(y=A) == BAD                             # the sum and the norm in one place
    assert call(rows=0, x=None, r=None, w=None, o=None, y=None, q=None, s=None) == moe.MOE_OK


def test_norm_gradient_refusals(lib):
    need = lib.moe_rms_norm_grad_scratch_bytes(4, 64)
    assert need >= 4 * 64 * 4 and lib.moe_rms_norm_grad_scratch_bytes(-1, 64) == -1
    assert lib.moe_rms_norm_grad_scratch_bytes(1 << 30, 64) == lib.moe_rms_norm_grad_scratch_bytes(1 << 20, 64)

    def call(rows=4, H=64, eps=1e-6, dy=A, dys=128, h=A, hs=128, w=A, ds=A, dss=128, dh=A, dhs=128, dw=A, ws=A, n=need):
        return lib.moe_rms_norm_grad(rows, H, eps, dy, dys, h, hs, w, ds, dss, dh, dhs, dw, ws, n, None)

    for name in ("dy", "h", "w", "dh", "ws"):
        assert call(**{name: None}) == BAD and call(**{name: A + 8}) == BAD, name
    assert call(ds=A + 8) == BAD and call(dw=A + 8) == BAD and call(n=need - 1) == BAD and call(ws=A + 16) == BAD
    for name in ("dys", "hs", "dss", "dhs"):
        assert call(**{name: 120}) == BAD and call(**{name: 136}) == BAD, name
    assert call(rows=-1) == BAD and call(H=12) == BAD and call(eps=0.0) == BAD


@pytest.mark.parametrize("name", ["moe_int8_pack", "moe_int8_unpack"])
def test_int8_rows_refusals(lib, name):
    def call(groups=1, rows=64, width=64, gated=0, x=A, xs=128, q=A, qs=64, s=A, ss=4, E=0, plan=None, ints=0):
        a = (x, xs, q, qs, s, ss) if name == "moe_int8_pack" else (q, qs, s, ss, x, xs)
        return getattr(lib, name)(groups, rows, width, gated, *a, E, plan, ints, None)

    assert call(groups=-1) == BAD and call(rows=-1) == BAD and call(width=0) == BAD and call(width=24) == BAD
    assert call(width=32784, xs=1 << 20, qs=1 << 20) == UNSUP and call(groups=1 << 30, rows=1 << 30) == UNSUP
    assert call(gated=2) == BAD and call(gated=1, rows=48) == BAD
    assert call(xs=120) == BAD and call(xs=136) == BAD and call(qs=48) == BAD and call(qs=72) == BAD
    assert call(ss=0) == BAD and call(ss=6) == BAD
    for arg in ("x", "q", "s"):
        assert call(**{arg: None}) == BAD and call(**{arg: A + 2}) == BAD, arg
    ints = 4 + 2 * 8
    assert call(E=8, plan=A, ints=ints - 1) == BAD and call(E=0, plan=A, ints=ints) == BAD
    assert call(E=8, plan=A + 4, ints=ints) == BAD
    assert call(E=8, plan=A, ints=ints, groups=2) == BAD and call(E=8, plan=A, ints=ints, gated=1) == BAD
    assert call(rows=0, x=None, q=None, s=None) == moe.MOE_OK


def test_int8_product_refusals(lib):
    def call(E=2, N=64, K=64, gated=0, wq=A, ws=A, xq=A, xst=64, xs=A, xss=4, rows=100, plan=A, ints=64, y=A, yst=128, err=None):
        return lib.moe_expert_product_int8(E, N, K, gated, wq, ws, xq, xst, xs, xss, rows, plan, ints, y, yst, err, None)

    assert call(E=0) == BAD and call(N=0) == BAD and call(K=0) == BAD
    assert call(N=48, yst=96) == BAD and call(K=40) == BAD and call(gated=2) == BAD
    assert call(E=4097, ints=1 << 20) == UNSUP and call(K=32784, xst=1 << 20) == UNSUP and call(N=65568, yst=1 << 20) == UNSUP
    assert call(rows=-1) == BAD and call(rows=1 << 31) == UNSUP
    assert call(yst=120) == BAD and call(yst=136) == BAD and call(gated=1, yst=48) == BAD
    assert call(xst=48) == BAD and call(xst=72) == BAD and call(xss=2) == BAD and call(xss=6) == BAD
    for name in ("wq", "ws", "xq", "xs", "y"):
        assert call(**{name: None}) == BAD and call(**{name: A + 2}) == BAD, name
    assert call(plan=A + 4) == BAD and call(ints=7) == BAD and call(err=A + 1) == BAD
    assert call(plan=None, ints=0) == BAD  # a dense layer has one expert
    assert call(rows=0, xq=None, xs=None, y=None) == moe.MOE_OK


def test_helpers_refuse_on_the_host(lib):
    """Tensors of another type, size, place or stride are refused before the library is called."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((64,), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_rms_norm(x, w, 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="expected x in"):
        moe.moe_rms_norm(x.float(), w, 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="unit column stride"):
        moe.moe_rms_norm(torch.zeros((64, 4), dtype=torch.bfloat16).t(), w, 1e-6, y=x)
    with pytest.raises(ValueError, match="scratch"):
        moe.moe_rms_norm_grad(x, x, w, 1e-6, x, dweight=torch.zeros(64))
    with pytest.raises(ValueError):
        moe.Int8Rows(33, 64, "cpu", gated=True)
    with pytest.raises(ValueError):
        moe.Int8Rows(32, 72, "cpu")
    with pytest.raises(ValueError, match="expected x of shape"):
        moe.Int8Rows(4, 64, "cpu").pack(torch.zeros((4, 32), dtype=torch.bfloat16))
    with pytest.raises(moe.MoeError):
        moe.Gate(moe.make_shape(1, 0, 4, 2, 64), "cpu")
    g = moe.Gate(moe.make_shape(1, 16, 4, 2, 64), "cpu")
    with pytest.raises(ValueError, match="expected logits in"):
        g.forward(torch.zeros((4, 16), dtype=torch.float16))
    with pytest.raises(ValueError, match="expected logits of shape"):
        g.forward(torch.zeros((4, 15)))
    with pytest.raises(ValueError, match="unit column stride"):
        g.forward(torch.zeros((1, 16)).expand(4, 16))  # rows on top of one another


def test_the_product_holds_tensors_to_their_sizes(lib):
    E, N, K, rows = 2, 64, 32, 5
    good = dict(wq=torch.zeros((E, N, K), dtype=torch.int8), ws=torch.zeros((E, N)), xq=torch.zeros((rows, K), dtype=torch.int8),
                xs=torch.zeros(rows), y=torch.zeros((rows, N), dtype=torch.bfloat16))

    def call(match, **k):
        a = {**good, **k}
        with pytest.raises(ValueError, match=match):
            moe.moe_expert_product_int8(E, N, K, 0, a["wq"], a["ws"], a["xq"], a["xs"], rows, None, a["y"], None)

    call("expected a CUDA tensor")
    call("wq", wq=torch.zeros((E, N, K - 1), dtype=torch.int8))
    call("wq", wq=torch.zeros((E, N, K)))
    on = lambda **k: {**{n: A for n in good}, **k}
    call("ws", **on(ws=torch.zeros((E, N - 1))))
    call("ws", **on(ws=torch.zeros((E, N), dtype=torch.float64)))
    call("xq", **on(xq=torch.zeros((rows - 1, K), dtype=torch.int8)))
    call("xq", **on(xq=torch.zeros((rows, K)).t()))
    call("xs", **on(xs=torch.zeros(rows - 1)))
    call("y", **on(y=torch.zeros((rows, N - 1), dtype=torch.bfloat16)))
    call("y", **on(y=torch.zeros((rows, N))))


def test_buffers_refuse_a_product_before_its_rows(lib):
    s = moe.make_shape(1, 4, 8, 2, 64, expert_alignment=128, quant=1)
    buf = moe.Buffers(s, "cpu")
    w = moe.Int8Rows(32, 64, "cpu", groups=4)
    y = torch.zeros((1, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="before the product"):
        buf.expert_product_int8(w, y)
    with pytest.raises(ValueError, match="weights of 4 experts"):
        buf.expert_product_int8(moe.Int8Rows(32, 48, "cpu", groups=4), y)
    with pytest.raises(ValueError, match="int8 payload"):
        moe.Buffers(moe.make_shape(1, 4, 8, 2, 64, expert_alignment=128), "cpu").expert_product_int8(w, y)
