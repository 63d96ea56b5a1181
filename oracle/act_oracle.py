"""CPU oracle of the 8-bit activation checkpoints, the RMS norm and the weight
gradient: plain numpy, written from the formulas in include/scape.h.  Codes
are exact; everything else is computed in binary64."""

import numpy as np

BLOCK = 32


def pack(x):
    """(codes int8 [rows][pitch], scales uint8 [rows][blocks]) of an fp32
    matrix."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    full = np.zeros((rows, nb * BLOCK), dtype=np.float64)
    full[:, :cols] = x
    blk = full.reshape(rows, nb, BLOCK)
    with np.errstate(invalid="ignore"):
        bad = ~np.isfinite(blk).all(axis=2)
    blk = np.where(bad[:, :, None], 0.0, blk)
    amax = np.abs(blk).max(axis=2)
    # least e >= -126 with amax <= 127 * 2^e
    _, ex = np.frexp(amax)  # amax = m * 2^ex, 1/2 <= m < 1, so e is ex - 7 or one more
    e = np.maximum(np.where(amax > np.ldexp(127.0, ex - 7), ex - 6, ex - 7), -126)
    q = np.rint(np.ldexp(blk, -e[:, :, None]))
    q = np.where((e == 122)[:, :, None], np.clip(q, -63, 63), q)  # 64 * 2^122 is no fp32 number
    s = np.where(bad, 255, np.where(amax == 0, 0, e + 127))
    q = np.where((s == 0)[:, :, None], 0, q)
    assert np.abs(q).max(initial=0) <= 127
    return q.astype(np.int8).reshape(rows, nb * BLOCK), s.astype(np.uint8)


def unpack(codes, scales, cols):
    """Values in binary64 (exact)."""
    rows = codes.shape[0]
    e = scales.astype(np.int64) - 127
    step = np.where(scales == 255, np.nan, np.where(scales == 0, 0.0, np.ldexp(1.0, e)))
    v = codes.astype(np.float64).reshape(rows, -1, BLOCK) * step[:, :, None]
    return v.reshape(rows, -1)[:, :cols]


def norm_sum(x, residual=None):
    """The fp32 sum that the norm is of."""
    x = np.asarray(x, dtype=np.float32)
    return x if residual is None else x + np.asarray(residual, dtype=np.float32)


def norm_rstd(hs, eps):
    """Binary64 reciprocal RMS of fp32 rows."""
    h = hs.astype(np.float64)
    return 1.0 / np.sqrt((h * h).mean(axis=1) + np.float64(np.float32(eps)))


def norm_forward(x, weight, eps, residual=None):
    """(y, rstd) in binary64, nothing rounded but the fp32 sum."""
    hs = norm_sum(x, residual)
    rs = norm_rstd(hs, eps)
    return hs.astype(np.float64) * rs[:, None] * np.asarray(weight, dtype=np.float64), rs


def norm_backward(dy, xh, rstd, weight, dres=None):
    """(dh, dweight) in binary64 from the normalised rows xh."""
    dy, xh = np.asarray(dy, dtype=np.float64), np.asarray(xh, dtype=np.float64)
    g = dy * np.asarray(weight, dtype=np.float64)
    dh = np.asarray(rstd, dtype=np.float64)[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    if dres is not None:
        dh = dh + np.asarray(dres, dtype=np.float64)
    return dh, (dy * xh).sum(axis=0)


def wgrad(dy, x, gain=None):
    """(dw [out][in], dbias [out]) in binary64."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    dw = dy.T @ x
    return (dw if gain is None else dw * np.asarray(gain, dtype=np.float64)), dy.sum(axis=0)
