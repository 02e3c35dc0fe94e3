"""The attention oracle against itself: closed forms and central differences (CPU)."""

import numpy as np
import pytest

from oracle import attention as A


@pytest.mark.parametrize("causal,window,nq,nk", [(False, 0, 5, 7), (True, 0, 6, 9), (True, 3, 8, 8), (True, 0, 5, 2)])
def test_attention_backward_is_the_difference_quotient(causal, window, nq, nk):
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(nq, 4, 6)), r.normal(size=(nk, 2, 6)), r.normal(size=(nk, 2, 6))
    g = r.normal(size=q.shape)
    grads = A.attention_backward(g, q, k, v, causal, window)
    for i, d in enumerate(grads):
        way = r.normal(size=d.shape)
        args = [[q, k, v], [q, k, v]]
        args[0][i] = args[0][i] + 1e-5 * way
        args[1][i] = args[1][i] - 1e-5 * way
        quotient = sum(s * (g * A.attention(*a, causal, window)[0]).sum() for s, a in zip((1, -1), args)) / 2e-5
        assert abs(quotient - (d * way).sum()) < 1e-7


def test_rows_without_keys_and_uniform_rows():
    out, lse = A.attention(np.ones((4, 1, 3)), np.zeros((2, 1, 3)), np.arange(6.0).reshape(2, 1, 3), causal=True)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()
    np.testing.assert_allclose(out[3, 0], [1.5, 2.5, 3.5])
    np.testing.assert_allclose(lse[2:, 0], [0.0, np.log(2.0)], atol=1e-15)
    assert A.allowed(3, 5, True, 2).sum(-1).tolist() == [2, 2, 2]


def test_norm_rope_backward_is_the_difference_quotient():
    r = np.random.default_rng(2)
    x, w, g = r.normal(size=(5, 3, 10)), r.normal(size=10), r.normal(size=(5, 3, 10))
    at, freq = np.arange(5) * 7, np.array([1.0, 0.1, 0.01])
    dx, dw = A.norm_rope_backward(g, x, w, at, freq, 1e-5)
    f = lambda x_, w_: (g * A.norm_rope(x_, w_, at, freq, 1e-5)).sum()
    wx, ww = r.normal(size=x.shape), r.normal(size=10)
    h = 1e-5
    assert abs((f(x + h * wx, w) - f(x - h * wx, w)) / (2 * h) - (dx * wx).sum()) < 1e-7
    assert abs((f(x, w + h * ww) - f(x, w - h * ww)) / (2 * h) - (dw * ww).sum()) < 1e-7
    # a rotation keeps the length of the normed head
    y = A.norm_rope(x, np.ones(10), at, freq, 1e-12)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-9)
