"""The plain forms of the embedding, the log probabilities and the clipping,
pinned against hand-worked values and central differences."""

import numpy as np
import pytest

from oracle import ends_oracle as E


def test_embed_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    pos = np.array([[0.5, -0.5]])
    got = E.embed([2, -1, 0, 3], table, 2.0, [0, 0, 1, -7], pos)
    assert np.array_equal(got, [[10.5, 11.5], [0.5, -0.5], [2.0, 4.0], [0.0, 0.0]])


def test_embed_backward_is_the_transpose():
    r = np.random.default_rng(1)
    ids = np.array([4, 0, 4, 9, -100, 2, 4, 5])
    dy = r.standard_normal((8, 3))
    d, mag, cnt = E.embed_backward(ids, dy, 5, 1.5)
    assert cnt.tolist() == [1, 0, 1, 0, 3]
    assert np.array_equal(d[1], np.zeros(3)) and np.array_equal(d[3], np.zeros(3))
    # <dy, embed(table)> = <dtable, table> for any table
    for _ in range(3):
        table = r.standard_normal((5, 3))
        assert np.isclose((dy * E.embed(ids, table, 1.5)).sum(), (d * table).sum(), rtol=1e-13)
    assert (mag >= np.abs(d)).all()


def test_log_probabilities_by_hand():
    x = np.log(np.array([[1.0, 2.0, 5.0], [1.0, 1.0, 2.0]]))
    assert np.allclose(np.exp(E.log_softmax(x)), [[0.125, 0.25, 0.625], [0.25, 0.25, 0.5]], rtol=1e-14)
    assert np.allclose(E.token_logp(x, [1, 5]), [np.log(0.25), 0.0], rtol=1e-14)
    assert np.isclose(E.entropy(x)[1], 1.5 * np.log(2), rtol=1e-14)
    assert np.allclose(np.exp(E.log_softmax(x[:1], 2.0)), [[1 / 30, 4 / 30, 25 / 30]], rtol=1e-14)
    ids, lp = E.top(np.array([[3.0, 7.0, 3.0, 7.0, 1.0]]), 4)
    assert ids.tolist() == [[1, 3, 0, 2]] and (np.diff(lp[0]) <= 0).all()
    # a row that is all but decided keeps its digits
    far = np.array([[50.0, 0.0, 0.0]])
    assert np.isclose(E.token_logp(far, [0])[0], -2 * np.exp(-50.0), rtol=1e-12)
    assert np.isclose(E.entropy(far)[0], 2 * 51 * np.exp(-50.0), rtol=1e-12)


def test_log_probabilities_of_special_rows():
    inf, nan = np.inf, np.nan
    x = np.array([[-inf, -inf], [0.0, -inf], [nan, 0.0], [inf, 0.0]])
    lp = E.log_softmax(x)
    assert np.array_equal(lp[0], [-inf, -inf]) and np.array_equal(lp[1], [0.0, -inf])
    assert np.isnan(lp[2:]).all()
    assert np.array_equal(E.entropy(x)[:2], [0.0, 0.0])
    assert np.array_equal(E.dlogits(x[:2], [0, 0], [1.0, 1.0], [1.0, 1.0]), np.zeros((2, 2)))
    assert np.array_equal(E.dlogits(x[2:], [0, -1], [0.0, 1.0]), np.zeros((2, 2)))  # weights of zero
    assert E.top(x[2:], 2)[0].tolist() == [[0, 1], [0, 1]]


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_dlogits_against_differences(scale):
    r = np.random.default_rng(2)
    x = r.standard_normal((3, 7)) * 2
    x[1, 3] = -np.inf
    y, w, d = [2, 0, 9], r.standard_normal(3), r.standard_normal(3)

    def loss(x):
        return (w * E.token_logp(x, y, scale) + d * E.entropy(x, scale)).sum()

    got = E.dlogits(x, y, w, d, scale)
    for i in range(3):
        for j in range(7):
            if np.isinf(x[i, j]):
                assert got[i, j] == 0.0
                continue
            hi, lo = x.copy(), x.copy()
            hi[i, j] += 1e-5
            lo[i, j] -= 1e-5
            # truncation h^2/6 * third derivative (below 20 here): 3e-10; rounding 1e-15 / h
            assert abs((loss(hi) - loss(lo)) / 2e-5 - got[i, j]) < 2e-9


def test_norm_and_clipping_by_hand():
    a, b = np.array([3.0, 0.0]), np.array([[4.0]])
    assert E.grad_norm([a, b]) == 5.0 and E.grad_norm([a, b], 0.5) == 2.5
    assert E.clip_factor(5.0, 1.0) == 0.2 and E.clip_factor(2.5, 1.0, 0.5) == 0.2
    assert E.clip_factor(5.0, 5.0) == 1.0 and E.clip_factor(5.0, np.inf, 0.5) == 0.5
    assert E.clip_factor(np.inf, 1.0, 0.5) == 0.5 and E.clip_factor(np.nan, 1.0) == 1.0
    assert E.grad_norm([np.array([1e200])]) == np.inf and E.grad_norm([np.array([np.float32(3e38)])]) > 2e38
