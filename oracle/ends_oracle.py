"""Plain numpy forms, in 64 bits, of the operators at the ends of a training
step: embedding and its gradient, log probabilities of given tokens with
entropy, alternatives and the gradient of the logits, norm and clipping.
Shares no code with the library."""

import numpy as np


# ---------------------------------------------------------------- embedding


def embed(ids, table, scale=1.0, pos=None, pos_table=None):
    """Rows [tokens][cols] of scale * table[ids] + pos_table[pos]; a number
    outside its table stands for zero."""
    out = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[t] = scale * table[v].astype(np.float64)
        if pos is not None and 0 <= pos[t] < pos_table.shape[0]:
            out[t] += pos_table[pos[t]].astype(np.float64)
    return out


def embed_backward(ids, dy, vocab, scale=1.0):
    """(dtable, magnitude, count): scale times the sum of each token's rows,
    the sum of their absolute values, and their number."""
    d = np.zeros((vocab, dy.shape[1]))
    mag = np.zeros_like(d)
    cnt = np.zeros(vocab, dtype=np.int64)
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            d[v] += dy[t].astype(np.float64)
            mag[v] += np.abs(dy[t].astype(np.float64))
            cnt[v] += 1
    return scale * d, abs(scale) * mag, cnt


# --------------------------------------------------------- log probabilities


def row_stats(x, scale=1.0):
    """(m, s) per row: the largest logit and log(1 + the sum over the other
    words of e^(scale (x - m))); a row of -inf has (-inf, 0), one with a NaN
    (NaN, NaN), one with +inf and no NaN (+inf, NaN)."""
    x = x.astype(np.float64)
    rows = x.shape[0]
    m, s = np.empty(rows), np.empty(rows)
    for r in range(rows):
        if np.isnan(x[r]).any():
            m[r] = s[r] = np.nan
            continue
        m[r] = x[r].max()
        if m[r] == -np.inf:
            s[r] = 0.0
        elif m[r] == np.inf:
            s[r] = np.nan
        else:
            rest = np.delete(x[r], int(x[r].argmax()))
            s[r] = np.log1p(np.exp((rest - m[r]) * scale).sum())
    return m, s


def log_softmax(x, scale=1.0):
    """Log probabilities [rows][vocab]; a row of -inf keeps -inf."""
    m, s = row_stats(x, scale)
    out = np.empty(x.shape)
    for r in range(x.shape[0]):
        if m[r] == -np.inf:
            out[r] = -np.inf
        elif np.isnan(s[r]):
            out[r] = np.nan
        else:
            out[r] = (x[r].astype(np.float64) - m[r]) * scale - s[r]
    return out


def token_logp(x, targets, scale=1.0):
    lp = log_softmax(x, scale)
    return np.array([lp[r, y] if 0 <= y < x.shape[1] else 0.0 for r, y in enumerate(targets)])


def plogp(lp):
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        return np.where(p == 0.0, 0.0, p * lp)


def entropy(x, scale=1.0):
    return -plogp(log_softmax(x, scale)).sum(axis=1)


def top(x, k, scale=1.0):
    """(ids, log probabilities) of the k likeliest words: by logit from the
    largest (NaN before all), equal ones by index."""
    lp = log_softmax(x, scale)
    ids = np.empty((x.shape[0], k), dtype=np.int64)
    for r in range(x.shape[0]):
        row = x[r].astype(np.float64)
        ids[r] = sorted(range(row.size), key=lambda j: (0, 0.0, j) if np.isnan(row[j]) else (1, -row[j], j))[:k]
    return ids, np.take_along_axis(lp, ids, axis=1)


def dlogits(x, targets, dlogp=None, dentropy=None, scale=1.0):
    """Gradient of sum dlogp * logp + dentropy * entropy."""
    rows, vocab = x.shape
    lp = log_softmax(x, scale)
    p = np.exp(lp)
    h = entropy(x, scale)
    out = np.zeros((rows, vocab))
    for r in range(rows):
        y = -1 if targets is None else targets[r]
        w = float(dlogp[r]) if dlogp is not None and 0 <= y < vocab else 0.0
        d = float(dentropy[r]) if dentropy is not None else 0.0
        if (w == 0.0 and d == 0.0) or (x[r] == -np.inf).all():
            continue
        out[r] = -w * p[r] - d * (plogp(lp[r]) + p[r] * h[r])
        if 0 <= y < vocab:
            out[r, y] += w
    return scale * out


# ------------------------------------------------------------ norm, clipping


def grad_norm(tensors, scale=1.0):
    """scale * the 2-norm over all tensors, as a Python float."""
    with np.errstate(invalid="ignore", over="ignore"):
        return float(scale * np.sqrt(sum(float((t.astype(np.float64) ** 2).sum()) for t in tensors)))


def clip_factor(norm, max_norm, scale=1.0):
    if not np.isfinite(norm) or norm <= max_norm:
        return float(scale)
    return float(scale) * (float(max_norm) / norm)
