"""The 64-bit references of the gate, the norm and int8 rows themselves: values worked out by hand, and differences."""

import numpy as np

from tests import router_ref as ref


def test_gate_by_hand():
    z = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [3.0, 3.0, 3.0, 1.0]]))
    z = np.vstack([z, np.full((1, 4), -np.inf), [[0.0, -np.inf, -np.inf, -np.inf]]])
    f = ref.gate(z, 2, balance=0.5)
    assert f["idx"].tolist() == [[2, 1], [0, 1], [-1, -1], [0, -1]]
    np.testing.assert_allclose(f["weights"], [[2 / 3, 1 / 3], [0.5, 0.5], [0, 0], [1, 0]])
    assert f["count"].tolist() == [2, 2, 1, 0, 3]
    prob = np.array([1 / 8 + 0.3 + 1, 1 / 4 + 0.3, 1 / 2 + 0.3, 1 / 8 + 0.1]) / 3
    np.testing.assert_allclose(f["prob"], prob)
    np.testing.assert_allclose(f["loss"], 0.5 * 4 * (np.array([2, 2, 1, 0]) / 6 * prob).sum())


def test_gate_gradient_is_the_differences():
    rng = np.random.default_rng(1)
    z, dw = rng.normal(size=(5, 7)), rng.normal(size=(5, 3))
    mask = np.array([1, 1, 0, 1, 1])
    for normalize in (True, False):
        args = dict(mask=mask, normalize=normalize, scale=2.5, balance=0.3)
        f = ref.gate(z, 3, **args)
        got, _ = ref.gate_grad(f, f["idx"], dw, 1.7, normalize, 2.5, 0.3)
        want = np.zeros_like(z)
        for g in range(5):
            for e in range(7):
                side = []
                for h in (1e-6, -1e-6):
                    zz = z.copy()
                    zz[g, e] += h
                    o = ref.gate(zz, 3, **args)
                    assert np.array_equal(o["idx"], f["idx"])
                    side.append((o["weights"] * dw).sum() + 1.7 * o["loss"])
                want[g, e] = (side[0] - side[1]) / 2e-6
        np.testing.assert_allclose(got, want, atol=1e-8)


def test_norm_gradient_is_the_differences():
    rng = np.random.default_rng(2)
    h, w, dy = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8))
    dh, dw, _, _ = ref.rms_grad(dy, h, w, 1e-3)
    loss = lambda h, w: (ref.rms(h, w, 1e-3)[0] * dy).sum()
    for at in np.ndindex(3, 8):
        d = np.zeros((3, 8))
        d[at] = 1e-6
        np.testing.assert_allclose(dh[at], (loss(h + d, w) - loss(h - d, w)) / 2e-6, atol=1e-8)
    for c in range(8):
        d = np.zeros(8)
        d[c] = 1e-6
        np.testing.assert_allclose(dw[c], (loss(h, w + d) - loss(h, w - d)) / 2e-6, atol=1e-8)


def test_int8_rows_by_hand():
    x = np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [np.inf, 1, 2, 3], [np.nan, 1, 2, 3]], np.float32)
    q, s = ref.int8_rows(x)
    assert q.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0], [0, 0, 0, 0], [0, 0, 0, 0]]
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3])
    assert ref.gated_order(64)[:4].tolist() == [0, 1, 2, 3] and ref.gated_order(64)[16] == 32


def test_product_by_hand():
    wq = np.array([[1, 2], [3, -4]], np.int8)
    xq = np.array([[5, 6]], np.int8)
    y, off = ref.product(wq, np.array([0.5, 2.0], np.float32), xq, np.array([3.0], np.float32), False)
    assert y.tolist() == [[17 * 1.5, -9 * 6.0]] and (off < 1e-4).all()
