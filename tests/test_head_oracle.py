"""Pins of the float64 reference of the dense operators (oracle/head.py): hand
values, identities and central differences.  No GPU."""

import numpy as np
import pytest

from oracle import head as oh


def _diff(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_rmsnorm_of_a_hand_example():
    y = oh.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    assert oh.q8_scale(y)[0] == pytest.approx(8 / np.sqrt(12.5) / 127, rel=1e-15)


# central differences of step 1e-5 are off by about 1e-10 (truncation) + 1e-11 (rounding) of values around 1
@pytest.mark.parametrize("n", [1, 2, 7])
def test_rmsnorm_gradient_against_differences(n):
    rng = np.random.default_rng(n)
    h, w, dy, dh = (rng.standard_normal(s) for s in ((3, n), (n,), (3, n), (3, n)))
    dx, dw = oh.rmsnorm_backward(dy, h, w, 1e-3, dh)
    f = lambda hh: np.sum(oh.rmsnorm(hh, w, 1e-3) * dy) + np.sum(hh * dh)  # noqa: E731
    np.testing.assert_allclose(dx, _diff(f, h), atol=1e-7)
    np.testing.assert_allclose(dw, _diff(lambda ww: np.sum(oh.rmsnorm(h, ww, 1e-3) * dy), w), atol=1e-7)


def test_logprobs_of_hand_examples():
    logp, H = oh.logprobs(np.array([[0.0, 0.0, 0.0, 0.0], [0.0, np.log(3.0), -np.inf, -np.inf],
                                    [-np.inf] * 4]))
    np.testing.assert_allclose(logp[0], np.log(0.25), rtol=1e-15)
    np.testing.assert_allclose(logp[1, :2], [np.log(0.25), np.log(0.75)], rtol=1e-15)
    assert np.isneginf(logp[1, 2:]).all() and np.isneginf(logp[2]).all()
    np.testing.assert_allclose(H, [np.log(4), -0.25 * np.log(0.25) - 0.75 * np.log(0.75), 0.0], rtol=1e-15)


def test_logprobs_of_rows_far_from_zero():
    """A row of a type's lowest value is a row of equals; nothing of it is lost in the sum with the maximum."""
    low = -3.402823466e38
    logp, H = oh.logprobs(np.full((1, 8), low))
    np.testing.assert_allclose(logp, np.log(1 / 8), rtol=1e-15)
    np.testing.assert_allclose(H, np.log(8), rtol=1e-15)


def test_top_takes_the_lowest_place_among_equals_and_nan_first():
    x = np.array([[1.0, 3.0, -0.0, 3.0, 0.0], [2.0, np.nan, np.inf, 2.0, np.nan]])
    np.testing.assert_array_equal(oh.top(x, 5), [[1, 3, 0, 2, 4], [1, 4, 2, 0, 3]])


def test_logprobs_gradient_against_differences():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 6))
    targets, dlp, dH = [1, 5, -100], rng.standard_normal(3), rng.standard_normal(3)
    idx, dtop = oh.top(x, 2), rng.standard_normal((3, 2))

    def f(v):
        logp, H = oh.logprobs(v)
        out = np.sum(H * dH) + np.sum(np.take_along_axis(logp, idx, 1) * dtop)
        return out + sum(dlp[i] * logp[i, t] for i, t in enumerate(targets) if t >= 0)

    got = oh.logprobs_backward(x, targets, dlp, dH, idx, dtop)
    np.testing.assert_allclose(got, _diff(f, x), atol=1e-7)
    np.testing.assert_allclose(got.sum(1), 0.0, atol=1e-12)   # adding a constant to a row changes nothing


def test_q8_linear_is_exact_on_whole_numbers():
    rng = np.random.default_rng(0)
    a, b = rng.integers(-127, 128, (4, 900)), rng.integers(-127, 128, (5, 900))
    want = np.array([[sum(int(p) * int(q) for p, q in zip(r, s)) for s in b] for r in a])
    np.testing.assert_array_equal(oh.q8_linear(a, np.ones(4), b, np.ones(5)), want)
