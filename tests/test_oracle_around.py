"""The fp64 forms of what stands around the experts, against closed forms,
differences and brute force (no GPU)."""
import numpy as np
import pytest

from oracle import around as oa


def test_layer_norm_closed_form():
    # a row of +-1 has mean 0 and variance 1
    x = np.array([[1.0, -1.0, 1.0, -1.0, 1.0, -1.0, 1.0, -1.0]])
    w, b = np.arange(8.0), np.full(8, 0.5)
    y, s, mean, rstd = oa.layer_norm(x, w, b, 3.0)
    assert mean[0] == 0 and rstd[0] == 0.5
    np.testing.assert_allclose(y[0], x[0] * 0.5 * w + 0.5, rtol=0, atol=0)
    y2, s2, _, _ = oa.layer_norm(x - 2.0, w, b, 3.0, residual=np.full((1, 8), 2.0))
    np.testing.assert_array_equal(y2, y)
    np.testing.assert_array_equal(s2, s)


@pytest.mark.parametrize("with_ds", [False, True])
def test_layer_norm_backward_against_differences(with_ds):
    rng = np.random.default_rng(5)
    T, d, eps = 5, 24, 1e-3
    x, w, b = rng.standard_normal((T, d)), rng.standard_normal(d), rng.standard_normal(d)
    dy, ds = rng.standard_normal((T, d)), rng.standard_normal((T, d)) if with_ds else None

    def loss(x_, w_, b_):
        y, s, _, _ = oa.layer_norm(x_, w_, b_, eps)
        return float((y * dy).sum() + (0 if ds is None else (s * ds).sum()))

    _, s, mean, rstd = oa.layer_norm(x, w, b, eps)
    dx, dw, db = oa.layer_norm_backward(dy, s, w, mean, rstd, ds)
    step = 1e-5
    for grad, at, put in ((dx, x, 0), (dw, w, 1), (db, b, 2)):
        for _ in range(12):
            v = rng.standard_normal(at.shape)
            args = [x, w, b]
            up, down = list(args), list(args)
            up[put], down[put] = at + step * v, at - step * v
            num = (loss(*up) - loss(*down)) / (2 * step)
            # central differences: the error is O(step^2) of third derivatives of order 10
            assert abs(num - float((grad * v).sum())) <= 1e-7 * (1 + abs(num))


def test_quantize_codes():
    q, s = oa.quantize(np.array([[127.0, -127.0, 63.4, 0.5, 1.5, -0.5, 0.0, 2.5]], dtype=np.float32))
    assert s[0] == 1.0
    np.testing.assert_array_equal(q[0], [127, -127, 63, 0, 2, 0, 0, 2])  # ties to even
    q, s = oa.quantize(np.zeros((1, 8), np.float32))
    assert s[0] == np.float32(2.0 ** -126) and not q.any()
    q, s = oa.quantize(np.array([[1.0, np.inf], [np.nan, 2.0], [1.0, 2.0]], np.float32))
    assert np.isnan(s[:2]).all() and not q[:2].any() and s[2] == np.float32(2) / np.float32(127)
    a = np.random.default_rng(1).standard_normal((40, 64)).astype(np.float32)
    q, s = oa.quantize(a)
    assert (np.abs(q.astype(int)).max(axis=1) == 127).all()
    # half a step, plus the two fp32 roundings on the way
    assert (np.abs(q * s[:, None].astype(np.float64) - a) <= s[:, None] * (0.5 + 127 * 2.0 ** -22)).all()


def test_kblocks_round_trip():
    q = np.random.default_rng(2).integers(-127, 128, (3, 5, 72)).astype(np.int8)
    b = oa.kblocks(q)
    assert b.shape == (3, 2, 5, 64) and not b[:, 1, :, 8:].any()
    assert b[1, 1, 3, 2] == q[1, 3, 66]
    np.testing.assert_array_equal(oa.from_kblocks(b, 72), q)


def test_int8_product_against_brute_force():
    rng = np.random.default_rng(3)
    q, w = rng.integers(-127, 128, (3, 9)).astype(np.int8), rng.integers(-127, 128, (4, 9)).astype(np.int8)
    s, ws = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32)
    got = oa.int8_product(q, s, w, ws)
    for r in range(3):
        for n in range(4):
            acc = sum(int(q[r, k]) * int(w[n, k]) for k in range(9))
            assert got[r, n] == acc * float(s[r]) * float(ws[n])


def test_norm_and_clip_factor():
    assert oa.grad_norm([np.array([3.0]), np.array([[4.0]])]) == 5.0
    assert oa.clip_factor(5.0, 10.0) == 1.0
    assert abs(oa.clip_factor(5.0, 1.0) - 0.2) < 1e-6
