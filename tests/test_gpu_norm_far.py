"""The norm and its gradient where the mean square and eps are near the end of binary32."""

import numpy as np
import pytest

from combine_moe_layout_02_gb300 import moe
from tests import router_ref as ref
from tests.test_gpu_norm import BF, U, _bf16, _np, _rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [16, 64, 1040, 7168])
@pytest.mark.parametrize("eps", [3.4e38, 1e38, 1e36, 1e-6])
def test_large_eps(H, eps):
    """eps counts next to squares whose sum leaves binary32, and where only the two together do."""
    import torch

    powers = [40, 58, 60, 61, 62, 63, 64, 66, 70, 100]
    x = _bf16((len(powers), H), 1) * torch.tensor([2.0 ** p for p in powers])[:, None].to(torch.bfloat16)
    w, dy = _bf16((H,), 2), _bf16((len(powers), H), 3)
    e32 = float(np.float32(eps))
    y, q, qs = torch.empty_like(x).cuda(), torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    moe.moe_rms_norm(x.cuda(), w.cuda(), eps, y=y, q=q, q_scale=qs)
    v, _ = ref.rms(_np(x), _np(w), e32)
    assert (np.abs(_np(y) - v) <= np.abs(v) * (BF + _rel(H) * (1 + BF)) + 1e-40).all()
    scale = np.abs(v).max(1) / 127
    assert (np.abs(_np(qs) - scale) <= scale * (_rel(H) + 2 * U)).all()
    assert (np.abs(_np(q) - v / scale[:, None]) <= 0.5 + 127 * (2 * _rel(H) + 4 * U)).all()
    dh = torch.empty_like(y)
    moe.moe_rms_norm_grad(dy.cuda(), x.cuda(), w.cuda(), eps, dh)
    want, _, mag, _ = ref.rms_grad(_np(dy), _np(x), _np(w), e32)
    # products of numbers of fewer bits near the end of binary32: as test_gpu_norm's rows of far values
    assert (np.abs(_np(dh) - want) <= np.abs(want) * BF + mag * (2 * _rel(H) + 80 * U) + 1e-37).all()


@pytest.mark.parametrize("H,rows", [(16, 4000), (128, 4000), (1040, 1000), (7168, 300)])
def test_codes_are_the_nearest(H, rows):
    """Of v's quotients themselves: the row's factor cancels, so a code is off by half and the two roundings of its quotient
    (three, and the scale's, where rows are normed first): 127 * 2^-22."""
    import torch

    x, r, w = _bf16((rows, H), 5), _bf16((rows, H), 6, 3.0), _bf16((H,), 7)
    x[-rows // 8:] *= 2.0 ** -80  # normed first
    r[-rows // 8:] *= 2.0 ** -80
    h = (x.float() + r.float()).double().numpy()  # binary32, as the sum is
    q, qs = torch.empty((rows, H), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_rms_norm(x.cuda(), w.cuda(), 1e-30, residual=r.cuda(), q=q, q_scale=qs)
    v = h * _np(w)
    quotient = v / (np.abs(v).max(1, keepdims=True) / 127)
    off = np.abs(_np(q) - quotient)
    assert off.max() <= 0.5 + 127 * 2.0 ** -22 <= 0.5 + 2.0 ** -15


def test_one_row_in_place_at_any_stride():
    """A single row has no next one: its strides mean nothing, in place either."""
    import torch

    x, w = _bf16((1, 64), 1).cuda(), _bf16((64,), 2).cuda()
    want, got = torch.empty_like(x), x.clone()
    moe.moe_rms_norm(x, w, 1e-6, y=want)
    p = got.data_ptr()
    assert moe.lib().moe_rms_norm(1, 64, 1e-6, p, 128, None, 0, w.data_ptr(), None, 0, p, 256, None, 0, None, 0, None) == moe.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    grads = [torch.empty_like(x), _bf16((1, 64), 3).cuda()]
    moe.moe_rms_norm_grad(grads[1], x, w, 1e-6, grads[0])
    p = grads[1].data_ptr()
    assert moe.lib().moe_rms_norm_grad(1, 64, 1e-6, p, 128, x.data_ptr(), 128, w.data_ptr(), None, 0, p, 256, None, None, 0, None) == moe.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(grads[1], grads[0])
