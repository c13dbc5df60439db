"""Pins of the float64 reference between the projections (oracle/attn.py): hand
values, identities and central differences.  No GPU."""

import numpy as np
import pytest

from oracle import attn as oa


def _diff(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_turn_of_a_hand_example():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    inv = np.array([np.pi / 2, np.pi])   # position 1: a quarter turn and a half turn
    np.testing.assert_allclose(oa.turn(x, [1], inv)[0, 0], [-3, -2, 1, -4, 5], atol=1e-15)
    np.testing.assert_allclose(oa.turn(x, [1], inv, True)[0, 0], [-2, 1, -3, -4, 5], atol=1e-15)
    np.testing.assert_allclose(oa.turn(oa.turn(x, [7], inv), [7], inv, sign=-1.0), x, atol=1e-14)


def test_scores_of_turned_heads_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k, inv = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), rng.random(4)
    a = np.sum(oa.turn(q, [5], inv) * oa.turn(k, [2], inv))
    b = np.sum(oa.turn(q, [105], inv) * oa.turn(k, [102], inv))
    assert a == pytest.approx(b, rel=1e-12)


# central differences of step 1e-5 are off by about 1e-10 (truncation) + 1e-11 (rounding) of values around 1
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_rope_gradient_against_differences(weighted, interleaved):
    rng = np.random.default_rng(1)
    x, dy, inv = rng.standard_normal((2, 3, 6)), rng.standard_normal((2, 3, 6)), rng.random(2)
    w = rng.random(6) + 0.5 if weighted else None
    f = lambda xx, ww: np.sum(oa.rope(xx, ww, [3, 9], inv, 1e-3, interleaved) * dy)  # noqa: E731
    dx, dw = oa.rope_backward(dy, x, w, [3, 9], inv, 1e-3, interleaved)
    np.testing.assert_allclose(dx, _diff(lambda v: f(v, w), x), atol=1e-7)
    if weighted:
        np.testing.assert_allclose(dw, _diff(lambda v: f(x, v), w), atol=1e-7)
    else:
        assert dw is None


def _paged(rng, lens, heads, dim, page, columns):
    pages = len(lens) * columns
    table = rng.permutation(pages).reshape(len(lens), columns)
    return rng.standard_normal((pages, heads, page, dim)), rng.standard_normal((pages, heads, page, dim)), table


def test_append_then_causal_attention_is_the_dense_one():
    rng = np.random.default_rng(2)
    starts, lens, scale = [0, 5, 5, 8], [5, 4, 9], 0.5
    kp, vp, table = _paged(rng, lens, 2, 4, 4, 3)
    k, v, q = rng.standard_normal((8, 2, 4)), rng.standard_normal((8, 2, 4)), rng.standard_normal((8, 4, 4))
    kp, vp = oa.append(kp, vp, k, v, starts, lens, table)
    out, lse = oa.attention(q, kp, vp, starts, lens, table, scale)
    for h in range(4):   # the first sequence is nothing but its rows
        s = scale * q[:5, h] @ k[:5, h // 2].T
        s[np.triu_indices(5, 1)] = -np.inf
        p = np.exp(s)
        np.testing.assert_allclose(out[:5, h], p @ v[:5, h // 2] / p.sum(1, keepdims=True), rtol=1e-12)
        np.testing.assert_allclose(lse[:5, h], np.log(p.sum(1)), rtol=1e-12)


def test_a_chain_is_a_tree_and_a_path_of_a_tree_is_a_chain():
    rng = np.random.default_rng(3)
    starts, lens, scale = [0, 6], [13], 0.7
    kp, vp, table = _paged(rng, lens, 1, 4, 8, 2)
    q = rng.standard_normal((6, 2, 4))
    chain = [(1 << (i + 1)) - 1 for i in range(6)]
    np.testing.assert_allclose(oa.attention(q, kp, vp, starts, lens, table, scale, chain)[0],
                               oa.attention(q, kp, vp, starts, lens, table, scale)[0], rtol=1e-13)
    # the path 0, 2, 5 of a tree, moved together, is a causal text of three rows
    tree = [0b1, 0b11, 0b101, 0b1001, 0b10011, 0b100101]
    got = oa.attention(q, kp, vp, starts, lens, table, scale, tree)[0][[0, 2, 5]]
    path = [[0, 2, 5, -1]]
    kp, vp = oa.accept(kp, path, starts, lens, table), oa.accept(vp, path, starts, lens, table)
    np.testing.assert_allclose(got, oa.attention(q[[0, 2, 5]], kp, vp, [0, 3], [10], table, scale)[0], rtol=1e-13)


def test_a_row_that_sees_nothing_is_zero():
    rng = np.random.default_rng(4)
    kp, vp, table = _paged(rng, [2], 1, 4, 8, 1)
    out, lse = oa.attention(rng.standard_normal((2, 1, 4)), kp, vp, [0, 2], [2], table, 1.0, [0, 0b10])
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1]).all()
