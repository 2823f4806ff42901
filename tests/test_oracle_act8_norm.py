"""The oracle's 8-bit blocks and layer norm against closed forms, brute force
and differences (CPU only)."""
import numpy as np
import pytest

from oracle import act8, norm


def test_e4m3_levels_and_nearest():
    assert act8.e4m3_value([0x00, 0x01, 0x08, 0x38, 0x7E, 0xFE]).tolist() == [0, 2 ** -9, 2 ** -6, 1.0, 448.0, -448.0]
    assert np.isnan(act8.e4m3_value([0x7F, 0xFF])).all()
    levels = act8.e4m3_value(np.arange(0x7F))
    assert np.array_equal(act8.e4m3_code(levels), np.arange(0x7F))
    rng = np.random.default_rng(0)
    q = np.concatenate([rng.uniform(-460, 460, 2000), rng.standard_normal(2000) * 2.0 ** rng.integers(-10, 4, 2000)])
    got = np.abs(act8.e4m3_value(act8.e4m3_code(q)))
    want = np.min(np.abs(np.minimum(np.abs(q), 448)[:, None] - levels[None, :]), axis=1)
    assert np.array_equal(np.abs(got - np.minimum(np.abs(q), 448)), want)
    # halfway between two levels: the even code
    mid = (levels[1:] + levels[:-1]) / 2
    lo = np.arange(0x7E)
    assert np.array_equal(act8.e4m3_code(mid), np.where(lo % 2 == 0, lo, lo + 1))


@pytest.mark.parametrize("fmt", act8.FORMATS)
def test_block_definition(fmt):
    rng = np.random.default_rng(1)
    X = np.float32(rng.standard_normal((40, 75)) * np.exp2(rng.integers(-30, 30, (40, 1))))
    codes, scales = act8.save(X, fmt)
    assert codes.shape == (40, 96) and scales.shape == (40, 3)
    assert not codes.reshape(40, 96)[:, 75:].any()
    back = act8.load(codes, scales, 75, fmt)
    for b in range(3):
        x, v = np.float64(X[:, 32 * b:32 * b + 32]), back[:, 32 * b:32 * b + 32]
        p = np.exp2(np.floor(np.log2(np.abs(x).max(1))))[:, None]
        if fmt == "mxint8":
            # half a step of p / 64, or saturation within one step
            assert np.all(np.abs(v - x) <= np.where(np.abs(x) > 126.5 / 64 * p, 1.0, 0.5) * p / 64)
        else:
            # half a unit in the last of 3 places, or of the subnormal step, or saturation at 1.75 p
            assert np.all(np.abs(v - x) <= np.maximum(np.where(np.abs(x) > 1.75 * p, 0.25 * p, np.abs(x) * 2.0 ** -4),
                                                      p / 256 * 2.0 ** -10))
    # what 8 bits hold is held again without a change
    c2, s2 = act8.save(back, fmt)
    assert np.array_equal(act8.load(c2, s2, 75, fmt), back)
    assert act8.amax(codes, scales, fmt) == np.abs(back).max()


@pytest.mark.parametrize("fmt", act8.FORMATS)
def test_special_blocks(fmt):
    X = np.zeros((5, 64), np.float32)
    X[0, 3], X[0, 40] = np.nan, 2.0
    X[1, 0], X[1, 33] = np.inf, -3.0
    X[2, 5] = np.float32(1e-45)
    X[3, 5] = np.finfo(np.float32).max
    codes, scales = act8.save(X, fmt)
    v = act8.load(codes, scales, 64, fmt)
    assert scales[0, 0] == scales[1, 0] == 255 and np.isnan(v[0, :32]).all() and np.isnan(v[1, :32]).all()
    assert v[0, 40] == 2.0 and v[1, 33] == -3.0
    assert not codes[0, :32].any() and scales[4].tolist() == [0, 0] and not v[4].any()
    assert v[2, 5] == 0 and scales[2, 0] == (7 if fmt == "mxint8" else 1)
    assert abs(v[3, 5] / X[3, 5] - 1) <= (2 ** -7 if fmt == "mxint8" else 2 ** -3)


def test_norm_backward_is_the_gradient():
    rng = np.random.default_rng(2)
    m, n, h = 5, 7, 1e-6
    x, dy = rng.standard_normal((m, n)) * 3 + 1, rng.standard_normal((m, n))
    w, b = rng.standard_normal(n), rng.standard_normal(n)
    _, mean, rstd = norm.forward(x, w, b)
    dx, dw, db = norm.backward(dy, x, mean, rstd, w)

    def loss(x, w, b):
        return float((dy * norm.forward(x, w, b)[0]).sum())

    for arr, grad, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        num = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            d = np.zeros_like(arr)
            d[i] = h
            args = [[x, w, b], [x, w, b]]
            args[0][at], args[1][at] = arr + d, arr - d
            num[i] = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        # central differences: h^2 of truncation, 2^-53 |loss| / h of rounding
        assert np.allclose(num, grad, rtol=0, atol=1e-7)


def test_norm_forward_normalises():
    rng = np.random.default_rng(3)
    y, mean, rstd = norm.forward(rng.standard_normal((9, 33)) * 5 - 2, eps=0.0)
    assert np.allclose(y.mean(1), 0, atol=1e-13) and np.allclose((y * y).mean(1), 1)
    y0, _, _ = norm.forward(np.full((2, 8), 3.0), w=np.full(8, 2.0), b=np.arange(8.0))
    assert np.array_equal(y0, np.tile(np.arange(8.0), (2, 1)))
