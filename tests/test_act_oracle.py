"""Pins of the activation oracle: the code format at its borders, the error
bound it promises, and the gradients against central differences."""

import numpy as np
import pytest

from oracle import act_oracle as A


def row(*v):
    return np.array([v], dtype=np.float32)


def test_codes_of_known_blocks():
    q, s = A.pack(row(127.0, -127.0, 0.5, 1.5, -2.5, 0.0))
    assert s.tolist() == [[127]]
    assert q[0, :6].tolist() == [127, -127, 0, 2, -2, 0] and not q[0, 6:].any()
    # just over 127 quanta takes the next scale
    q, s = A.pack(row(np.nextafter(np.float32(127.0), np.float32(200.0)), 3.0))
    assert s.tolist() == [[128]] and q[0, :2].tolist() == [64, 2]
    q, s = A.pack(row(1.0))
    assert s.tolist() == [[121]] and q[0, 0] == 64  # quantum 2^-6
    assert A.pack(row(0.0, -0.0))[1].tolist() == [[0]]


def test_codes_of_extreme_values():
    big = np.float32(np.finfo(np.float32).max)
    q, s = A.pack(row(big, -1.0))
    assert s.tolist() == [[249]] and q[0, :2].tolist() == [63, 0]
    q, s = A.pack(row(np.float32(2.0 ** -149)))
    assert s.tolist() == [[1]] and q[0, 0] == 0  # quantum 2^-126 is the least
    for bad in (np.inf, -np.inf, np.nan):
        q, s = A.pack(np.array([[1.0] * 40 + [bad]], dtype=np.float32))
        assert s[0, 1] == 255 and s[0, 0] == 121 and not q[0, 32:].any()
        v = A.unpack(q, s, 41)
        assert np.isnan(v[0, 32:]).all() and (v[0, :32] == 1.0).all()


@pytest.mark.parametrize("seed", [0, 1])
def test_error_is_at_most_half_a_quantum(seed):
    r = np.random.default_rng(seed)
    x = (r.standard_normal((50, 333)) * np.exp(4 * r.standard_normal((50, 1)))).astype(np.float32)
    q, s = A.pack(x)
    v = A.unpack(q, s, 333)
    quantum = np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, axis=1)[:, :333]
    assert (np.abs(v - x) <= quantum / 2).all()
    full = np.zeros((50, 352))
    full[:, :333] = x
    amax = np.repeat(np.abs(full).reshape(50, 11, 32).max(axis=2), 32, axis=1)[:, :333]
    # one scale lower 127 quanta do not reach amax: amax > 63.5 quanta
    assert (np.abs(v - x) <= amax / 127.0).all()


def test_error_bound_at_each_scale():
    """Half a quantum at every scale but the largest; 1/127 of the block's
    largest magnitude between the lowest scale and the largest."""
    r = np.random.default_rng(9)
    mant = r.uniform(1.0, 2.0, (256, 1))
    for lo in (-149, -135, -128, -126, -121, -120, 0, 100, 127):
        x = (r.uniform(-1.0, 1.0, (256, 32)) * mant * 2.0 ** lo).clip(-3.4e38, 3.4e38).astype(np.float32)
        q, s = A.pack(x)
        err = np.abs(A.unpack(q, s, 32) - x).max(axis=1)
        amax = np.abs(x).max(axis=1).astype(np.float64)
        quantum = np.ldexp(1.0, s[:, 0].astype(np.int64) - 127)
        low, top = s[:, 0] <= 1, s[:, 0] == 249
        assert (err[~top] <= quantum[~top] / 2).all() and (err[top] <= 1.5 * quantum[top]).all()
        assert (err[~low & ~top] <= amax[~low & ~top] / 127.0).all()
        assert (err[low] <= 2.0 ** -127).all()
        if lo <= -128:  # the relative bound ends there: everything is lost
            assert low.all() and (err == amax).all()
    x = np.linspace(0, float(np.finfo(np.float32).max), 32, dtype=np.float64).astype(np.float32)[None]
    q, s = A.pack(x)
    assert s.tolist() == [[249]] and (np.abs(A.unpack(q, s, 32) - x) <= 1.5 * 2.0 ** 122).all()


def test_values_are_exact_in_bf16():
    r = np.random.default_rng(3)
    q, s = A.pack((r.standard_normal((64, 64)) * 10.0 ** r.uniform(-30, 30, (64, 1))).astype(np.float32))
    v = A.unpack(q, s, 64).astype(np.float32)
    assert not (v.view(np.uint32) & 0xffff).any()


def test_norm_gradients_against_differences():
    r = np.random.default_rng(5)
    rows, cols, eps = 3, 7, 1e-5
    x = r.standard_normal((rows, cols)).astype(np.float32).astype(np.float64)
    w, dy = r.standard_normal(cols), r.standard_normal((rows, cols))

    def loss(x, w):
        rs = 1.0 / np.sqrt((x * x).mean(axis=1) + np.float64(np.float32(eps)))
        return (dy * (x * rs[:, None] * w)).sum()

    y, rs = A.norm_forward(x, w, eps)
    dh, dw = A.norm_backward(dy, x * rs[:, None], rs, w)
    d = 1e-5
    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(x)
            e[i, j] = d
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - dh[i, j]) < 1e-7
    for j in range(cols):
        e = np.zeros(cols)
        e[j] = d
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - dw[j]) < 1e-7


def test_weight_gradient_against_differences():
    r = np.random.default_rng(6)
    x, w, b = r.standard_normal((5, 4)), r.standard_normal((3, 4)), r.standard_normal(3)
    gain, dy = r.standard_normal(4), r.standard_normal((5, 3))
    dw, db = A.wgrad(dy, x, gain)
    loss = lambda w, b: (dy * ((x * gain) @ w.T + b)).sum()  # noqa: E731
    for o in range(3):
        for i in range(4):
            e = np.zeros_like(w)
            e[o, i] = 1e-4
            assert abs((loss(w + e, b) - loss(w - e, b)) / 2e-4 - dw[o, i]) < 1e-9
        e = np.zeros(3)
        e[o] = 1e-4
        assert abs((loss(w, b + e) - loss(w, b - e)) / 2e-4 - db[o]) < 1e-9
