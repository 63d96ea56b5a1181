"""The embedding, the log probabilities and the clipping on the GPU against
their plain 64-bit forms, within bounds counted from the roundings of each
formula: u = 2^-24 for a 32-bit operation, half an epsilon for the final
rounding to the output's type, n u times the sum of the absolute terms for a
32-bit sum of n terms in any order, and 4 u for exp, log1p and expm1."""

import numpy as np
import pytest

from oracle import ends_oracle as E

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {t: torch.finfo(t).eps / 2 for t in DT.values()}
# half of the spacing of the type's subnormal numbers: what rounding loses there
LEAST = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def S():
    from sparse_communication_distributed_amd import scape
    scape.lib()
    return scape


class Guarded:
    """A [rows][cols] matrix inside a larger buffer of sentinels."""

    def __init__(self, rows, cols, dtype, pad=0, lead=0, fill=None):
        ld = cols + pad
        self.buf = torch.full((rows * ld + lead + 64,), -77, dtype=dtype, device=DEV)
        self.t = self.buf[lead:lead + rows * ld].view(rows, ld)[:, :cols]
        self.lead, self.rows, self.ld = lead, rows, ld
        if fill is not None:
            self.t.copy_(torch.from_numpy(np.asarray(fill)))

    def check(self):
        rest = self.buf.clone()
        rest[self.lead:self.lead + self.rows * self.ld].view(self.rows, self.ld)[:, :self.t.shape[1]] = -77
        assert (rest == -77).all(), "written outside the matrix"


def f64(t):
    return t.double().cpu().numpy()


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def scratch(n):
    assert n > 0
    return torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)  # contents do not matter


def within(got, want, tol, name):
    got = f64(got) if torch.is_tensor(got) else got
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol)
    bad &= ~(got == want) & ~(np.isnan(got) & np.isnan(want))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} beyond the bound; first {i}: got {got[i]!r} "
                             f"want {want[i]!r} tolerance {np.broadcast_to(tol, bad.shape)[i]!r}")


# ---------------------------------------------------------------- embedding


def some_ids(count, vocab, seed, none=0.1):
    r = np.random.default_rng(seed)
    ids = np.minimum((vocab * r.random(count) ** 3).astype(np.int64), vocab - 1)
    away = np.array([-1, -100, vocab, vocab + 7])
    return np.where(r.random(count) < none, away[r.integers(0, 4, count)], ids)


@pytest.mark.parametrize("table_dt", list(DT))
@pytest.mark.parametrize("out_dt", list(DT))
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (3, 7, 31), (1, 100, 2048), (130, 50, 33), (2, 9, 4097),
                                               (700, 300, 64)])
def test_embed(S, tokens, vocab, cols, table_dt, out_dt):
    r = np.random.default_rng(tokens + cols)
    tt, ot = DT[table_dt], DT[out_dt]
    for bits, pad, lead, scale, npos in ((64, 0, 0, 1.0, 0), (32, 5, 3, -13.25, 11), (64, 8, 1, 0.3, 4)):
        it = torch.int64 if bits == 64 else torch.int32
        table = Guarded(vocab, cols, tt, pad, lead, r.standard_normal((vocab, cols)))
        pt = Guarded(npos, cols, tt, 2 * pad, 0, r.standard_normal((npos, cols))) if npos else None
        ids = some_ids(tokens, vocab, tokens)
        pos = some_ids(tokens, npos, 5) if npos else None
        if bits == 64:
            ids[-1] = (1 << 32)  # no token, though its lower half would be one
        out = Guarded(tokens, cols, ot, pad, lead)
        S.embed(dev(ids, it), table.t, out.t, scale=scale, pos=dev(pos, it) if npos else None,
                pos_table=pt.t if npos else None)
        scale = float(np.float32(scale))
        a = E.embed(ids, f64(table.t), scale)
        want = E.embed(ids, f64(table.t), scale, pos, f64(pt.t) if npos else None)
        tol = U * np.abs(a) + U * (np.abs(want) + U * np.abs(a)) + 3 * LEAST[ot]
        if ot != torch.float32:
            tol = tol + HALF[ot] * (np.abs(want) + 2 * U * (np.abs(a) + np.abs(want)))
        within(out.t, want, tol, "out")
        out.check()


def test_embed_by_value(S):
    """Rows come back as they are: whole rows of one type, special values."""
    for t in DT.values():
        table = torch.randn(5, 67, device=DEV).to(t)
        table[1, 3], table[1, 66], table[2, 0], table[2, 1] = INF, -INF, NAN, -0.0
        ids = torch.tensor([2, 1, 4, 1, 0], device=DEV)
        out = torch.empty(5, 67, dtype=t, device=DEV)
        S.embed(ids.view(5, 1), table, out)  # ids of any shape
        assert torch.equal(out.nan_to_num(7.0), table[ids].nan_to_num(7.0))


def test_embed_far_rows(S):
    """Rows further from the table's start than 2^32 bytes."""
    ld = (1 << 30) + 3
    table = torch.empty(4 * ld, dtype=torch.bfloat16, device=DEV).view(4, ld)[:, :40]
    table.copy_(torch.randn(4, 40, device=DEV))
    ids = torch.tensor([3, 0, 2, 3, -1], device=DEV, dtype=torch.int32)
    out = torch.full((5 * ld,), 3.0, dtype=torch.bfloat16, device=DEV).view(5, ld)
    S.embed(ids, table, out[:, :40])
    assert torch.equal(out[:4, :40], table[ids[:4].long()]) and (out[4, :40] == 0).all() and (out[:, 40:64] == 3).all()


BACK_SHAPES = [(1, 1, 1), (7, 5, 33), (300, 50, 777), (1531, 4099, 64), (5000, 7, 130), (2049, 3, 1280),
               (4097, 70000, 8), (64, 33, 2056), (20000, 900, 24), (1024, 1024, 40), (1025, 1, 16), (100, 300, 5000)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("tokens,vocab,cols", BACK_SHAPES)
def test_embed_backward(S, tokens, vocab, cols, dt):
    t = DT[dt]
    r = np.random.default_rng(tokens)
    for bits, pad, lead, scale, acc in ((64, 0, 0, 1.0, False), (32, 3, 1, -2.75, True)):
        it = torch.int64 if bits == 64 else torch.int32
        ids = some_ids(tokens, vocab, cols)
        if bits == 64 and tokens > 1:
            ids[1] = (3 << 32) + vocab // 2  # no token, though its lower half would be one
        dy = Guarded(tokens, cols, t, pad, lead, r.standard_normal((tokens, cols)))
        away = dev((ids < 0) | (ids >= vocab), torch.bool)
        dy.t.masked_fill_(away[:, None], NAN)  # of no token: not read
        old = r.standard_normal((vocab, cols)).astype(np.float32)
        out = Guarded(vocab, cols, torch.float32, 0, lead, old)
        S.embed_backward(dev(ids, it), dy.t, out.t, scratch(S.embed_workspace_bytes(tokens, cols)), scale=scale,
                         accumulate=acc)
        want, mag, cnt = E.embed_backward(ids, f64(dy.t), vocab, scale)
        n = cnt[:, None]
        tol = (n + 2) * U * (1 + n * U) * mag
        if acc:
            want = want + old
            # an fma a row may add to what is there: its roundings are of sums that hold the old value
            tol = np.where(n > 0, tol + (n + 1) * U * np.abs(old), 0.0)
        within(out.t, want, tol, "dtable")
        out.check()


@pytest.mark.parametrize("tokens", [1, 64, 1000, 3000, 40000])
def test_embed_backward_one_word(S, tokens):
    """All tokens the same word, and all of them padding: whole numbers, whose
    sums are exact in any order."""
    dy = torch.randint(-3, 4, (tokens, 72), device=DEV).to(torch.bfloat16)
    out = torch.full((9, 72), 5.0, device=DEV)
    ws = scratch(S.embed_workspace_bytes(tokens, 72))
    S.embed_backward(torch.full((tokens,), 4, device=DEV), dy, out, ws)
    want = torch.zeros(9, 72, device=DEV)
    want[4] = dy.float().sum(0)
    assert torch.equal(out, want)
    S.embed_backward(torch.full((tokens,), -100, device=DEV), dy, out, ws, accumulate=True)
    assert torch.equal(out, want)
    S.embed_backward(torch.full((tokens,), 9, device=DEV), dy, out, ws)
    assert (out == 0).all()


@pytest.mark.parametrize("tokens,vocab,cols", [(30000, 200, 96), (70000, 60000, 16), (9000, 40, 520),
                                               (131073, 3000, 24), (300000, 70, 8), (70000, 65536, 16),
                                               (300000, 20000, 8), (600, 1 << 24, 1), (5000, 300000, 40), (16384, 500000, 8),
                                               (16385, 9, 8), (3000, 1 << 22, 2), (600000, 262144, 1),
                                               (2200000, 40000, 1)])
def test_embed_backward_exact_and_repeatable(S, tokens, vocab, cols):
    g = torch.Generator(DEV).manual_seed(tokens)
    ids = (vocab * torch.rand(tokens, device=DEV, generator=g) ** 4).long()
    whole = torch.randint(-8, 9, (tokens, cols), device=DEV, generator=g).to(torch.bfloat16)
    ws = scratch(S.embed_workspace_bytes(tokens, cols))
    out = torch.empty(vocab, cols, device=DEV)
    S.embed_backward(ids, whole, out, ws)
    want = torch.zeros(vocab, cols, dtype=torch.float64, device=DEV).index_add_(0, ids, whole.double())
    assert torch.equal(out.double(), want)
    # any numbers: the same bits every time, from a workspace of any contents
    dy = torch.randn(tokens, cols, device=DEV, generator=g)
    S.embed_backward(ids, dy, out, ws)
    first = out.clone()
    for i in range(3):
        ws.fill_(i * 85)
        S.embed_backward(ids.int(), dy, out, ws)
        assert torch.equal(out, first)


def test_embed_empty(S):
    table, none = torch.randn(5, 8, device=DEV), torch.empty(0, 8, device=DEV)
    no_ids = torch.empty(0, dtype=torch.int64, device=DEV)
    S.embed(no_ids, table, none)
    out = torch.full((5, 8), 3.0, device=DEV)
    ws = scratch(S.embed_workspace_bytes(0, 8))
    S.embed_backward(no_ids, none, out, ws, accumulate=True)
    assert (out == 3).all()
    S.embed_backward(no_ids, none, out, ws)
    assert (out == 0).all()


# --------------------------------------------------------- log probabilities


def logits_of(rows, vocab, seed, kind):
    """fp64 logits: spread rows, and as `kind` says special ones among them."""
    r = np.random.default_rng(seed)
    x = 2.5 * r.standard_normal((rows, vocab)) + 4 * r.standard_normal((rows, 1))
    for i in range(rows):
        if i % 4 == 1:
            x[i, r.integers(vocab)] += 25.0  # all but decided
        if i % 4 == 2:
            x[i] = np.round(x[i])  # ties
        if kind == "masked" and i % 3 == 0:
            x[i, r.random(vocab) < 0.9] = -np.inf
    if kind == "special":
        for i in range(rows):
            j = r.integers(vocab)
            if i % 8 == 0:
                x[i] = -np.inf
            elif i % 8 == 1:
                x[i, j] = np.nan
            elif i % 8 == 2:
                x[i, j] = np.inf
            elif i % 8 == 3:
                x[i] = 1.25  # all equal
            elif i % 8 == 4:
                x[i] = -np.inf
                x[i, j] = -60000.0  # one word left
            elif i % 8 == 5:
                x[i] = -65504.0  # the lowest fp16, then the lowest of the type below
            elif i % 8 == 6:
                x[i] = np.where(r.random(vocab) < 0.5, -0.0, 0.0)
    return x


class Bounds:
    """Error bounds of a row's outputs, from the roundings along the formulas:
    t = scale (x - m) has three (difference, product, the constant), e^t four
    more of its own."""

    def __init__(self, x, scale):
        with np.errstate(all="ignore"):
            self.m, self.s = E.row_stats(x, scale)
            self.t = np.where(x == -np.inf, -np.inf, (x - self.m[:, None]) * scale)
            self.lp = E.log_softmax(x, scale)
            self.h = E.entropy(x, scale)
            t = np.where(np.isfinite(self.t), np.abs(self.t), 0.0)
            e = np.nan_to_num(np.exp(self.t))
            others = e.copy()
            others[np.arange(len(x)), np.nanargmax(np.nan_to_num(x, nan=-np.inf), axis=1)] = 0.0
            # a sum's own roundings: a workgroup of at least 64 threads sums the vocabulary's share of each one
            # after the other, then the threads' sums
            deep = x.shape[1] / 64 + 24
            o = others.sum(1)
            do = (others * (4 * U * t + 4 * U)).sum(1) + deep * U * o + x.shape[1] * 2.0 ** -126
            self.ds = do / (1 + o) + 4 * U * np.nan_to_num(self.s)
            self.dt = 4 * U * t
            self.dlp = self.dt + self.ds[:, None] + U * np.nan_to_num(np.abs(self.lp), posinf=0.0)
            u = (e * t).sum(1)
            du = (e * t * (4 * U * t + 10 * U)).sum(1) + deep * U * u + x.shape[1] * 2.0 ** -118
            self.dh = self.ds + du / (1 + o) + u / (1 + o) * (do / (1 + o) + 3 * U) + U * np.nan_to_num(self.h)

    def gradient(self, x, y, w, d, scale, dtype):
        want = E.dlogits(x, y, w, d, scale)
        rows, vocab = x.shape
        p = np.nan_to_num(np.exp(self.lp))
        lp = np.where(np.isfinite(self.lp), self.lp, 0.0)
        rel = self.dlp + 4 * U + 2 * U * np.abs(lp)
        w = np.zeros(rows) if w is None else np.abs(w.astype(np.float64))
        d = np.zeros(rows) if d is None else np.abs(d.astype(np.float64))
        tol = w[:, None] * p * (rel + 3 * U)
        for r in range(rows):
            if y is not None and 0 <= y[r] < vocab:
                j = y[r]
                tol[r, j] = w[r] * (p[r, j] * self.dlp[r, j] + 8 * U * abs(np.expm1(lp[r, j])))
        h = np.nan_to_num(self.h)[:, None]
        inner = np.abs(lp + h)
        ent = d[:, None] * p * (inner * (rel + 5 * U) + self.dlp + self.dh[:, None] + U * h)
        tol = scale * (tol + ent + 2 * U * (w[:, None] * p + d[:, None] * p * inner))
        tol = tol + np.nan_to_num(np.abs(want)) * (2 * U + HALF[dtype]) + 4 * LEAST[dtype] + scale * (w + d)[:, None] * 2.0 ** -118
        return want, tol


def check_logprobs(S, x, dt, targets, scale=1.0, top=0, pad=0, lead=0, bits=64, weights=True, ent=True, separate=False,
                   in_place=False):
    t = DT[dt]
    rows, vocab = x.shape
    a = Guarded(rows, vocab, t, pad, lead, x)
    x = f64(a.t)
    scale = float(np.float32(scale))
    r = np.random.default_rng(rows + vocab)
    it = torch.int64 if bits == 64 else torch.int32
    ty = dev(targets, it)
    v = lambda *s: Guarded(int(np.prod(s[:-1])), s[-1], torch.float32, 0, 2)  # noqa: E731
    logp, stats, h = v(1, rows), v(rows, 2), v(1, rows)
    top_lp, top_ids = (v(rows, top), Guarded(rows, top, torch.int32, 0, 3)) if top else (None, None)
    w = (r.standard_normal(rows) * (r.random(rows) < 0.9)).astype(np.float32) if weights else None
    d = (r.standard_normal(rows) * (r.random(rows) < 0.7)).astype(np.float32) if ent else None
    g = a if in_place else Guarded(rows, vocab, t, pad + 1, lead)
    ws = scratch(S.token_logprobs_workspace_bytes(rows, vocab, top))
    kw = dict(dlogp=None if w is None else dev(w), dentropy=None if d is None else dev(d))
    grad = weights or ent
    fused = dict(kw, dlogits=g.t) if grad and not separate else {}
    S.token_logprobs(a.t, ty, logp.t.view(-1), ws, stats=stats.t, entropy=h.t.view(-1),
                     top_logp=top_lp.t if top else None, top_ids=top_ids.t if top else None, scale=scale, **fused)
    if separate:
        S.token_logprobs_backward(a.t, ty, stats.t, g.t, entropy=h.t.view(-1), scale=scale, **kw)
    b = Bounds(x, scale)
    rows_ = np.arange(rows)
    there = (targets >= 0) & (targets < vocab)
    y = np.where(there, targets, 0)
    within(logp.t[0], E.token_logp(x, targets, scale), np.where(there, b.dlp[rows_, y], 0.0), "logp")
    # NaN rows hold NaN in stats; the largest logit of the others is exact
    within(stats.t[:, 0], b.m, np.zeros(rows), "m")
    within(stats.t[:, 1], b.s, b.ds, "log-sum")
    within(h.t[0], b.h, b.dh, "entropy")
    if top:
        ids, lp = E.top(x, top, scale)
        assert np.array_equal(top_ids.t.cpu().numpy(), ids), "alternatives"
        within(top_lp.t, lp, np.take_along_axis(b.dlp, ids, 1), "top_logp")
    if grad:
        want, tol = b.gradient(x, targets, w, d, scale, t)
        within(g.t, want, tol, "dlogits")
    for m in (a, logp, stats, h, top_lp, top_ids, g):
        if m is not None:
            m.check()


VOCABS = [1, 2, 7, 8, 9, 64, 100, 255, 257, 1000, 2048, 4099, 8192, 16385, 32000, 50257, 65537, 131077, 300001]


def some_targets(rows, vocab, x, seed):
    r = np.random.default_rng(seed)
    y = np.where(r.random(rows) < 0.4, np.nan_to_num(x, nan=-np.inf).argmax(1), r.integers(0, vocab, rows))
    if rows > 2:
        y[r.integers(rows)] = -100
        y[r.integers(rows)] = vocab
    return y


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("vocab", VOCABS)
def test_token_logprobs(S, vocab, dt):
    rows = 9 if vocab < 5000 else 4
    for i, (kind, pad, lead, bits, scale) in enumerate((("plain", 0, 0, 64, 1.0), ("masked", 3, 1, 32, 0.6))):
        x = logits_of(rows, vocab, vocab + i, kind)
        check_logprobs(S, x, dt, some_targets(rows, vocab, x, vocab), scale, top=min(vocab, (5, 64)[i]), pad=pad,
                       lead=lead, bits=bits, separate=i == 1)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("vocab", [3, 64, 777, 4096, 32000, 140001])
def test_token_logprobs_special_rows(S, vocab, dt):
    """Rows of -inf, NaN, +inf, one value, one word, the lowest values, zeros of both signs."""
    rows = 17 if vocab < 5000 else 8
    x = logits_of(rows, vocab, 3, "special")
    y = some_targets(rows, vocab, x, 9)
    for separate in (False, True):
        check_logprobs(S, x, dt, y, 1.0 if separate else 1.5, top=min(vocab, 33), separate=separate)


@pytest.mark.parametrize("weights,ent", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("rows,vocab", [(1, 32000), (700, 129), (37, 2500), (2, 200003)])
def test_token_logprobs_parts(S, rows, vocab, weights, ent):
    x = logits_of(rows, vocab, rows, "masked")
    y = some_targets(rows, vocab, x, 1)
    for dt, separate, in_place in (("bf16", False, False), ("fp32", weights or ent, False), ("fp16", False, True),
                                   ("fp32", weights or ent, True)):
        if in_place and not (weights or ent):
            continue
        check_logprobs(S, x, dt, y, 1.0, weights=weights, ent=ent, separate=separate, in_place=in_place)


def test_token_logprobs_many_rows(S):
    """More rows than a launch's workgroups take at once, and as many as a step has."""
    for rows, vocab, dt in ((70000, 33, "fp32"), (5000, 1000, "bf16")):
        x = logits_of(rows, vocab, 5, "masked")
        check_logprobs(S, x, dt, some_targets(rows, vocab, x, 2), top=3)


def test_token_logprobs_ties(S):
    """Equal logits everywhere: alternatives by index, whatever the number of equal ones."""
    for vocab, dt in ((64, "bf16"), (5000, "fp32"), (50257, "fp16"), (100003, "bf16"), (200001, "fp32")):
        x = np.zeros((5, vocab))
        x[1] = np.random.default_rng(1).integers(0, 3, vocab)  # three values
        x[2, vocab // 3:] = 1.0
        x[3, -1] = 2.0
        x[4] = -np.inf
        x[4, vocab // 2] = 0.0
        check_logprobs(S, x, dt, np.zeros(5, dtype=np.int64), top=64)


def test_token_logprobs_outputs_alone(S):
    """Each output alone is what it is among the others; no targets where none are needed."""
    x = dev(logits_of(6, 4100, 8, "masked"), torch.bfloat16)
    y = torch.arange(6, device=DEV)
    ws = scratch(S.token_logprobs_workspace_bytes(6, 4100, 7))
    mk = lambda: dict(stats=torch.full((6, 2), 9.0, device=DEV), entropy=torch.full((6,), 9.0, device=DEV),  # noqa: E731
                      top_logp=torch.full((6, 7), 9.0, device=DEV),
                      top_ids=torch.full((6, 7), 9, dtype=torch.int32, device=DEV))
    logp, full = torch.empty(6, device=DEV), mk()
    S.token_logprobs(x, y, logp, ws, **full)
    alone = torch.empty(6, device=DEV)
    S.token_logprobs(x, y, alone, ws)
    assert torch.equal(alone, logp)
    for name in full:
        part = mk()
        S.token_logprobs(x, None, None, ws, **{name: part[name]})
        assert torch.equal(part[name], full[name]), name
    g, h = torch.empty_like(x), torch.empty_like(x)
    w = torch.randn(6, device=DEV)
    S.token_logprobs(x, y, None, ws, dlogp=w, dlogits=g)
    S.token_logprobs(x, y, logp, ws, dlogp=w, dlogits=h, **full)
    assert torch.equal(g, h)


def test_token_logprobs_masked_rows_are_not_read(S):
    """Rows of no weight may hold anything and get zeros."""
    x = torch.full((4, 900), NAN, device=DEV)
    x[2] = torch.randn(900, device=DEV)
    y = torch.tensor([-100, 3, 5, -100], device=DEV)
    w = torch.tensor([1.0, 0.0, 1.0, INF], device=DEV)
    g, logp = torch.full_like(x, 7.0), torch.empty(4, device=DEV)
    ws = scratch(S.token_logprobs_workspace_bytes(4, 900, 0))
    S.token_logprobs(x, y, logp, ws, dlogp=w, dlogits=g)
    assert (g[[0, 1, 3]] == 0).all() and torch.isfinite(g[2]).all() and g[2].abs().sum() > 0
    assert logp[0] == 0 and logp[1].isnan() and logp[3] == 0


def test_token_logprobs_far_rows_and_empty(S):
    ld = (1 << 29) + 5
    x = torch.empty(9 * ld, dtype=torch.bfloat16, device=DEV).view(9, ld)[:, :70]  # the last past 2^32 elements
    small = torch.randn(9, 70, device=DEV).bfloat16()
    x.copy_(small)
    y, w = torch.arange(9, device=DEV), torch.randn(9, device=DEV)
    ws = scratch(S.token_logprobs_workspace_bytes(9, 70, 4))
    # A row's sums are grouped by where its 16-byte borders lie, so bits are alike where rows begin alike: every
    # 77 logits as every ld (both 5 past a multiple of 8).  Beside `small`, whose rows begin otherwise, a sum may
    # have rounded in another order; each form is within the bound counted for a sum in any order.
    assert ld % 8 == 77 % 8 and x.data_ptr() % 16 == 0
    alike = torch.empty(9 * 77, dtype=torch.bfloat16, device=DEV).view(9, 77)[:, :70]
    alike.copy_(small)
    assert alike.data_ptr() % 16 == 0
    b = Bounds(f64(small), 1.0)
    want, tol = b.gradient(f64(small), np.arange(9), f64(w), None, 1.0, torch.bfloat16)
    res = []
    for m in (x, alike, small):
        logits = f64(m)
        logp, ids = torch.empty(9, device=DEV), torch.empty(9, 4, dtype=torch.int32, device=DEV)
        S.token_logprobs(m, y, logp, ws, top_ids=ids, dlogp=w, dlogits=m)
        res.append((logp, ids, m.clone()))
        within(logp, E.token_logp(logits, np.arange(9), 1.0), b.dlp[np.arange(9), np.arange(9)], "logp")
        within(m, want, tol, "dlogits")
    assert all(torch.equal(a, b) for a, b in zip(*res[:2]))
    assert torch.equal(res[0][1], res[2][1])
    none = torch.empty(0, 70, device=DEV)
    S.token_logprobs(none, y[:0], logp[:0], scratch(S.token_logprobs_workspace_bytes(0, 70, 0)))
    S.token_logprobs_backward(none, y[:0], torch.empty(0, 2, device=DEV), none, dlogp=w[:0])


# ------------------------------------------------------------ norm, clipping

SIZES = [[1], [7], [4096], [2048, 2048], [1, 0, 3, 8191, 16, 77777], [0, 0, 0], [5] * 300, [300000, 1, 2049] * 2]


def place(sizes, dtype, lead):
    """Tensors of a buffer at odd places, sentinels between them."""
    buf = torch.full((sum(sizes) + 9 * len(sizes) + 64,), -77.0, dtype=dtype, device=DEV)
    at, out = lead, []
    for n in sizes:
        out.append(buf[at:at + n])
        at += n + 9
    return buf, out


@pytest.mark.parametrize("dt,out_dt", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"),
                                       ("fp16", "fp32")])
@pytest.mark.parametrize("sizes", SIZES)
def test_clip(S, sizes, dt, out_dt):
    t, ot = DT[dt], DT[out_dt]
    r = np.random.default_rng(len(sizes))
    for groups in {1, len(sizes) if len(sizes) < 5 else 2}:
        if len(sizes) % groups:
            continue
        for scale, max_norm, lead in ((1.0, 1.0, 0), (0.37, 40.0, 3), (8.0, INF, 1), (1.0, 1e6, 5)):
            _, grads = place(sizes, t, lead)
            for g in grads:
                g.copy_(dev(r.standard_normal(g.numel()) * np.exp(r.standard_normal())))
            src = [f64(g) for g in grads]
            buf, outs = place(sizes, ot, lead + 1)
            gl = S.GradList(grads, out=outs, groups=groups)
            ws = scratch(S.grad_workspace_bytes(gl))
            norm, n2 = torch.full((groups,), -7.0, device=DEV), torch.full((groups,), -7.0, device=DEV)
            S.grad_norm(gl, norm, ws, scale=scale)
            S.clip_grads(gl, max_norm, n2, ws, scale=scale)
            assert torch.equal(norm, n2)
            fs, per = float(np.float32(scale)), len(sizes) // groups
            for i in range(groups):
                want = E.grad_norm(src[i * per:(i + 1) * per], fs)
                within(norm[i:i + 1], np.array([want]), want * U * (1 + 1e-6), "norm")
                f = E.clip_factor(want, max_norm, fs)
                for j in range(i * per, (i + 1) * per):
                    v = src[j] * f
                    within(outs[j], v, np.abs(v) * HALF[ot] * (1 + 1e-6) + LEAST[ot], "clipped")
            inside = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
            for o in outs:
                inside[o.storage_offset():o.storage_offset() + o.numel()] = True
            assert (buf[~inside] == -77).all(), "written outside the tensors"
            # in place, the same
            own = S.GradList(grads, groups=groups)
            S.clip_grads(own, max_norm, n2, ws, scale=scale)
            assert torch.equal(norm, n2)
            if ot == t:
                assert all(torch.equal(g, o) for g, o in zip(grads, outs))


def test_clip_special_values(S):
    big = torch.tensor([3e38, -3e38, 1e30], device=DEV)
    tiny = torch.tensor([1e-44, 2e-44, 0.0], device=DEV)
    bad = torch.tensor([1.0, INF, -2.0], device=DEV)
    nan = torch.tensor([NAN, 2.0, 4.0], device=DEV)
    for g, norm, want in ((big, INF, None), (tiny, float(np.float32(np.sqrt(5) * 1e-44)), tiny * 0.5), (bad, INF, bad * 0.5),
                          (nan, NAN, nan * 0.5)):
        gl, out = S.GradList([g]), torch.empty_like(g)
        gl = S.GradList([g], out=[out])
        n = torch.zeros(1, device=DEV)
        S.clip_grads(gl, 1.0, n, scratch(S.grad_workspace_bytes(gl)), scale=0.5)
        if g is big:  # squares of such gradients pass fp32's range, their norm does not
            assert np.isclose(n.item(), np.sqrt(2) * 1.5e38, rtol=1e-6)
            assert np.isclose(f64(out), np.array([1, -1, 1 / 3e8]) / np.sqrt(2), rtol=1e-6).all()
        else:
            assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0))
            if g is not tiny:
                assert (n.item() == norm) or (n.isnan().item() and np.isnan(norm))
    # a factor of 1: the very same bits (a NaN's among them)
    g = torch.randn(5000, device=DEV)
    g[17] = -0.0
    want = g.clone()
    gl = S.GradList([g])
    S.clip_grads(gl, 1e9, n, scratch(S.grad_workspace_bytes(gl)))
    assert torch.equal(g.view(torch.int32), want.view(torch.int32))


def test_clip_long_and_many(S):
    """A tensor past 2^32 bytes, more tensors than a launch takes, more groups than a launch takes."""
    g = torch.ones((1 << 30) + 12345, device=DEV)
    gl = S.GradList([g])
    n = torch.zeros(1, device=DEV)
    S.clip_grads(gl, 2.0, n, scratch(S.grad_workspace_bytes(gl)))
    root = np.sqrt(g.numel())
    assert abs(n.item() - root) <= U * root * (1 + 1e-6)
    assert abs(g.min().item() - 2 / root) <= U * 2 / root * (1 + 1e-6) and g.min() == g.max()
    del g, gl
    grads = [torch.full((i % 5,), float(i % 7), device=DEV, dtype=torch.bfloat16) for i in range(700)]
    gl = S.GradList(grads, groups=350)
    n = torch.full((350,), -1.0, device=DEV)
    S.grad_norm(gl, n, scratch(S.grad_workspace_bytes(gl)))
    want = [E.grad_norm([f64(grads[2 * i]), f64(grads[2 * i + 1])]) for i in range(350)]
    within(n, np.array(want), np.array(want) * U * (1 + 1e-6), "norms")
    # groups far apart in one launch: all but a few tensors are empty
    some = {3: 2.0, 4100: 3.0, 9000: 5.0}
    grads = [torch.full((2,) if i in some else (0,), some.get(i, 0.0), device=DEV) for i in range(10000)]
    gl = S.GradList(grads, groups=10000)
    n = torch.full((10000,), -1.0, device=DEV)
    S.clip_grads(gl, 1.0, n, scratch(S.grad_workspace_bytes(gl)))
    want = torch.zeros(10000, dtype=torch.float64)
    for i, v in some.items():
        want[i] = v * 2 ** 0.5
        assert (grads[i] - 2 ** -0.5).abs().max() < 1e-7
    within(n, want.numpy(), want.numpy() * U * (1 + 1e-6), "norms")


def test_optimizer_clips_each_worker(S):
    """ScapeOptimizer.step with max_norm is a step on rows clipped one by one."""
    from sparse_communication_distributed_amd import workload as W
    cfg = W.flat_config("clip", 4 * 5000, 4, 2, "0.9")
    w0 = dev(W.init_params(cfg))
    a, b = (S.ScapeOptimizer(w0.clone(), cfg.P, cfg.K, cfg.k) for _ in range(2))
    for t in range(1, 4):
        g = dev(W.grads(cfg, t))
        g[0] *= 100.0
        limit = 1.5 * E.grad_norm([f64(g[1])])
        plain = g.clone()
        a.step(g, max_norm=limit)
        f = E.clip_factor(E.grad_norm([f64(plain[0])]), float(np.float32(limit)))
        assert f < 1 and torch.equal(g[1], plain[1])
        clipped = dev(f64(plain[0]) * f, torch.float64).float()
        assert (g[0] - clipped).abs().max() <= 2 * U * clipped.abs().max()
        within(a.grad_norm, np.array([E.grad_norm([f64(p)]) for p in plain]), 1e-3, "norms")
        b.step(g)
        for name in ("params", "m", "v", "e"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
