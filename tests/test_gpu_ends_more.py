"""More of the embedding, the log probabilities and the clipping on the GPU:
where results are held to single roundings, long sums, and the borders of the
kernels' variants."""

import numpy as np
import pytest

from oracle import ends_oracle as E

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
U = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module")
def S():
    from sparse_communication_distributed_amd import scape
    scape.lib()
    return scape


def scratch(n):
    assert n > 0
    return torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)  # contents do not matter


# ------------------------------------------------------------------ clipping

# binary digits, the exponent of the least quantum, the largest number
FORMAT = {torch.bfloat16: (8, -133, 2.0 ** 128 - 2.0 ** 120), torch.float16: (11, -24, 65504.0)}


def nearest(x, t):
    """The values of type t next to binary64 numbers, ties to even."""
    digits, least, most = FORMAT[t]
    _, e = np.frexp(x)
    q = np.ldexp(1.0, np.maximum(e - digits, least))
    r = np.rint(x / q) * q  # q is a power of two: exact but for rint
    return np.where(np.abs(r) > most, np.copysign(INF, x), r)


@pytest.mark.parametrize("t", list(FORMAT))
def test_clipped_values_are_rounded_once(S, t):
    """Every finite 16-bit number times 24-bit factors (products that 53 bits
    hold): the nearest 16-bit number, also where the product lies so close to the
    middle of two that its fp32 value is the middle."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(t).to(DEV)
    x = x[torch.isfinite(x)]
    v = x.double().cpu().numpy()
    norm = torch.zeros(1, device=DEV)
    missed = 0
    for f in (0.5730769038200378, 0.47821101546287537, 0.153273805975914, 0.831818163394928, 1.3618420362472534, 3.7e-5,
              300.0 / 7):
        f = float(np.float32(f))
        want = nearest(v * f, t)
        with np.errstate(over="ignore"):
            missed += (nearest((v * f).astype(np.float32).astype(np.float64), t) != want).sum()
        for src, out in ((x, torch.empty_like(x)), (x.clone(), None)):
            gl = S.GradList([src], out=None if out is None else [out])
            S.clip_grads(gl, INF, norm, scratch(S.grad_workspace_bytes(gl)), scale=f)
            got = (src if out is None else out).double().cpu().numpy()
            assert np.array_equal(got, want), (f, np.flatnonzero(got != want)[:5])
    assert missed > 100  # factors at which a second rounding shows


@pytest.mark.parametrize("in_place", [True, False])
def test_clip_of_gradients_whose_squares_fp32_loses(S, in_place):
    """Subnormal gradients, clipped to a tenth of their norm, and the largest,
    whose small neighbour is far below them: norm and values within a rounding of
    the 64-bit ones."""
    for values, share, scale in (([1e-40, 2e-40, 0.0], 0.1, 0.5), ([1e-30, -3e-30, 2e-31], 0.3, 1.0),
                                 ([3e38, -3e38, 1e30], 2.0 ** -127, 0.5)):
        g = torch.tensor(values, device=DEV)
        v = g.double().cpu().numpy()
        want = E.grad_norm([v], scale)
        assert 0 < want < 3.4e38
        limit = float(np.float32(share * want))
        out = g if in_place else torch.full_like(g, 7.0)
        gl = S.GradList([g], out=None if in_place else [out])
        n = torch.full((1,), -1.0, device=DEV)
        ws = scratch(S.grad_workspace_bytes(gl))
        S.grad_norm(gl, n, ws, scale=scale)
        assert abs(n.item() - want) <= max(want * U * (1 + 1e-6), 2.0 ** -150)
        n.fill_(-1.0)
        S.clip_grads(gl, limit, n, ws, scale=scale)
        assert abs(n.item() - want) <= max(want * U * (1 + 1e-6), 2.0 ** -150)
        clipped = v * E.clip_factor(want, limit, scale)
        got = out.double().cpu().numpy()
        assert (np.abs(got - clipped) <= np.maximum(np.abs(clipped) * U * (1 + 1e-6), 2.0 ** -150)).all(), (got, clipped)
        assert got[0] != 0


def test_grad_norm_of_lists_that_overlap(S):
    """Lists whose tensors share memory: clipping refuses them, the norm, which
    only reads, counts each as it is."""
    buf, other = torch.randn(100, device=DEV), torch.randn(100, device=DEV)
    a, b, c = buf[:40], buf[40:80], buf[30:50]
    n, ws = torch.zeros(1, device=DEV), scratch(1 << 16)
    for gl in (S.GradList([a, a]), S.GradList([a, b, c]), S.GradList([a], out=[buf[1:41]]),
               S.GradList([buf, other[:4]], out=[other, buf[20:24]])):
        with pytest.raises(ValueError, match="overlaps another tensor"):
            S.clip_grads(gl, 1.0, n, ws)
        S.grad_norm(gl, n, ws)
        want = E.grad_norm([g.double().cpu().numpy() for g in gl.grads])
        assert abs(n.item() - want) <= want * U * (1 + 1e-6)


@pytest.mark.parametrize("sizes", [[16], [8, 8], [1] * 200 + [16] * 200])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip_by_a_norm_past_fp32(S, sizes, in_place):
    """Finite gradients whose norm is no fp32 number: clipped by that norm, which
    is written as infinite.  Beside them a group with an infinity: scaled alone."""
    grads = [torch.full((n,), 3e38, device=DEV) for n in sizes] + [torch.full((n,), 2.0, device=DEV) for n in sizes]
    grads[len(sizes)][0] = INF
    outs = None if in_place else [torch.empty_like(g) for g in grads]
    gl = S.GradList(grads, out=outs, groups=2)
    norm = torch.zeros(2, device=DEV)
    S.clip_grads(gl, 8.0, norm, scratch(S.grad_workspace_bytes(gl)), scale=0.5)
    got = torch.cat(grads if in_place else outs).double().cpu().numpy()
    n = sum(sizes)
    assert norm[0] == INF and norm[1] == INF  # 0.5 x 3e38 x 4 and more
    want = 8.0 / n ** 0.5
    assert np.abs(got[:n] - want).max() <= want * 2.0 ** -23  # a rounding, and those of the factor in 64 bits
    assert got[n] == INF and (got[n + 1:] == 1.0).all()


# ----------------------------------------------------------------- embedding


def table_of(ids, dy, vocab):
    """The sums of whole numbers dy [tokens][cols] (host) by word, on the device; ids may hold -1."""
    return torch.from_numpy(np.stack([np.bincount(ids + 1, weights=column, minlength=vocab + 1)[1:] for column in dy.T],
                                     axis=1)).to(DEV)


@pytest.mark.parametrize("tokens,cols,depth", [(1 << 20, 8, 64), (1 << 18, 8, 64), (200001, 320, 150)])
def test_embed_backward_frequent_word_keeps_its_digits(S, tokens, cols, depth):
    """All tokens one word, all rows one number: roundings that all go one way,
    so the error grows with the number of additions behind one another.  Those of
    a chunk of 32, of an eighth of a part's partial rows, in pairs and of the
    parts are `depth` at most."""
    for value in (1.1, 0.3, 1.7):
        dy = torch.full((tokens, cols), value, device=DEV)
        value = float(np.float32(value))
        out = torch.empty(2, cols, device=DEV)
        ws = scratch(S.embed_workspace_bytes(tokens, cols))
        S.embed_backward(torch.zeros(tokens, dtype=torch.int64, device=DEV), dy, out, ws)
        want = tokens * value
        off = (out[0].double().cpu().numpy() / want - 1) / U
        assert np.abs(off).max() <= depth, off
        assert (out[1] == 0).all()


@pytest.mark.parametrize("tokens,cols", [(70000, 4), (70000, 20), (40000, 130), (30000, 300), (600000, 9), (9000, 1030)])
def test_embed_backward_runs_of_every_length(S, tokens, cols):
    """Words with 0 to thousands of partial rows in turn, at every place among the
    chunks: whole numbers, whose sums are exact in any order."""
    r = np.random.default_rng(cols)
    sizes = [tokens // 3, 1, 511, 512, 513, 40, 8 * 64 + 7, 8 * 65, 16 * 64 - 1, 16 * 65 + 9, 32 * 17, 32 * 64 + 33,
             32 * 66, 7, 2]
    sizes = [s for s in sizes if s < tokens // 2]
    while sum(sizes) < tokens:
        sizes.append(int(min(tokens - sum(sizes), np.exp(r.uniform(0, np.log(4000))))))
    cut = np.cumsum(sizes)
    sizes = sizes[:int(np.searchsorted(cut, tokens, side="right"))]
    word = np.repeat(np.arange(len(sizes)), sizes)
    word = np.concatenate([word, np.full(tokens - word.size, len(sizes))])
    word = r.permutation(word)
    ids = torch.from_numpy(word).to(DEV)
    vocab = len(sizes) + 3
    whole = r.integers(-8, 9, (tokens, cols))
    dy = torch.from_numpy(whole).to(DEV).to(torch.bfloat16)
    want = table_of(word, whole, vocab)
    out = torch.full((vocab, cols), 2.0, device=DEV)
    ws = scratch(S.embed_workspace_bytes(tokens, cols))
    S.embed_backward(ids, dy, out, ws, scale=0.5)
    assert torch.equal(out.double(), 0.5 * want)
    S.embed_backward(ids, dy, out, ws, accumulate=True, scale=0.5)
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("tokens,vocab", [(37888, 1000), (37889, 1000), (36864, 32000), (36865, 32000), (30720, 131072),
                                          (30721, 131072), (24001, 60000)])
def test_embed_backward_where_the_sort_changes(S, tokens, vocab):
    """As many tokens as the sort's lists hold and one more; every word's sum
    exact, and all tokens one word, which fills the lists of one workgroup."""
    r = np.random.default_rng(tokens)
    whole = r.integers(-8, 9, (tokens, 9))
    dy = torch.from_numpy(whole).to(DEV).to(torch.bfloat16)
    out = torch.empty(vocab, 9, device=DEV)
    ws = scratch(S.embed_workspace_bytes(tokens, 9))
    some = (vocab * r.random(tokens) ** 2).astype(np.int64)
    some[r.random(tokens) < 0.1] = -1
    for ids in (some, np.full(tokens, vocab - 1), np.arange(tokens) % vocab):
        t = torch.from_numpy(ids).to(DEV)
        want = table_of(ids, whole, vocab)
        S.embed_backward(t, dy, out, ws)
        assert torch.equal(out.double(), want)
        ws.fill_(0xA5)
        S.embed_backward(t.int(), dy, out, ws)
        assert torch.equal(out.double(), want)


@pytest.mark.parametrize("vocab,cols", [(24400, 1024), (24590, 1024), (24001, 1021), (25001, 1021), (2000000, 13)])
def test_embed_backward_clears_large_tables(S, vocab, cols):
    """Rows of no token are zero, at tables on both sides of the size from which
    they are cleared past the caches; those beside the table stay."""
    tokens, lead = 300, 5
    r = np.random.default_rng(vocab)
    ids = r.integers(0, vocab, tokens)
    ids[:100] = np.arange(100) * 3
    ids[-1] = vocab - 1
    whole = r.integers(-8, 9, (tokens, cols))
    dy = torch.from_numpy(whole).to(DEV).to(torch.bfloat16)
    buf = torch.full((vocab * cols + 64,), 7.0, device=DEV)
    out = buf[lead:lead + vocab * cols].view(vocab, cols)
    S.embed_backward(torch.from_numpy(ids).to(DEV), dy, out, scratch(S.embed_workspace_bytes(tokens, cols)))
    words, place = np.unique(ids, return_inverse=True)
    sums = table_of(place, whole, words.size)
    there = torch.from_numpy(words).to(DEV)
    assert torch.equal(out[there].double(), sums)
    out[there] = 0
    assert (buf[:lead] == 7).all() and (buf[lead + vocab * cols:] == 7).all() and not out.any()


# --------------------------------------------------------- log probabilities


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [1, 5, 900, 1031, 4099, 33001, 70001])
def test_token_logprobs_rows_of_no_weight(S, vocab, t):
    """A row without a weight gets zeros from either call, in place or not, into
    rows that begin anywhere, whatever its logits and stats are; its neighbours
    keep their gradients, and nothing beside the rows is written."""
    rows, lead = 6, 3
    x = torch.randn(rows, vocab, device=DEV)
    y = torch.arange(rows, device=DEV) % vocab
    w = torch.tensor([1.0, 0.0, -2.0, 0.0, 0.0, 0.5], device=DEV)
    d = torch.tensor([0.0, 0.0, 1.0, 0.0, 0.0, 0.0], device=DEV)
    y[3] = -100
    w[3] = INF  # of no token: no weight
    none = torch.tensor([1, 3, 4], device=DEV)
    ws = scratch(S.token_logprobs_workspace_bytes(rows, vocab, 0))
    x = x.to(t)
    bare = x.clone()
    bare[1], bare[3], bare[4] = float("nan"), INF, float("nan")
    logp, h, stats = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV)
    for ent in (None, d):
        res = []
        for logits in (x, bare):
            for fused in (True, False):
                for in_place in (False, True):
                    ld = vocab + 5
                    buf = torch.full((rows * ld + 16,), 7.0, dtype=t, device=DEV)
                    out = buf[lead:lead + rows * ld].view(rows, ld)[:, :vocab]
                    src = logits
                    if in_place:
                        out.copy_(logits)
                        src = out
                    kw = dict(dlogp=w, dentropy=ent)
                    S.token_logprobs(src, y, logp, ws, stats=stats, entropy=h, **(dict(kw, dlogits=out) if fused else {}))
                    if not fused:
                        S.token_logprobs_backward(src, y, stats, out, entropy=h, **kw)
                    assert (out[none] == 0).all(), (fused, in_place)
                    res.append(out[[0, 2, 5]].double())
                    inside = torch.zeros_like(buf, dtype=torch.bool)
                    inside[lead:lead + rows * ld].view(rows, ld)[:, :vocab] = True
                    assert (buf[~inside] == 7).all()
        if vocab > 1:
            assert all(torch.isfinite(r).all() and r.abs().sum() > 0 for r in res)
        # the logits beside a row change nothing in it
        for a, b in zip(res[:4], res[4:]):
            assert torch.equal(a, b)


# --------------------------------------------------------------------- lists


def test_grad_list_whose_tensors_moved(S):
    """Tensors given other memory: the list goes on with its own, and what the
    program allocates since is left as it is."""
    a, row = torch.full((100000,), 2.0, device=DEV), torch.zeros(100000, device=DEV)
    norm = torch.full((1,), -1.0, device=DEV)
    for gl in (S.GradList([a]), S.GradList([a], out=[row])):
        ws = scratch(S.grad_workspace_bytes(gl))
        kept = a.detach()
        a.data = torch.full((100000,), 5.0, device=DEV)
        if gl.out:
            row.data = torch.zeros(100000, device=DEV)
        del kept  # the list alone holds the old memory
        new = [torch.full((100000,), 7.0, device=DEV) for _ in range(6)]
        S.clip_grads(gl, INF, norm, ws, scale=0.25)
        assert (a == 5).all() and (row == 0).all() and all((t == 7).all() for t in new)
        S.grad_norm(gl, norm, ws)
        if gl.out is None:
            assert abs(norm.item() / (0.5 * 100000 ** 0.5) - 1) < 1e-6
        a.data = torch.full((100000,), 2.0, device=DEV)
    # a new list takes the new memory
    S.clip_grads(S.GradList([a], out=[row]), INF, norm, ws, scale=2.0)
    assert (row == 4).all() and (a == 2).all()


# ----------------------------------------------------------------- optimizer


def test_refused_step_leaves_the_gradients(S):
    """A step that is refused for its hyper-parameters, its gradients or its limit
    has clipped nothing and counted nothing; put right, it is the step it would
    have been."""
    from sparse_communication_distributed_amd import workload as W
    cfg = W.flat_config("refused", 4 * 5000, 4, 2, "0.9")
    w0 = torch.from_numpy(W.init_params(cfg)).to(DEV)
    a, b = (S.ScapeOptimizer(w0.clone(), cfg.P, cfg.K, cfg.k, count_nonfinite=True) for _ in range(2))
    g = torch.from_numpy(W.grads(cfg, 1)).to(DEV)
    g[1, 3] = INF
    limit = 0.5 * float(g[0].norm())
    lr, bt = a.lr, a.bt

    def bad_lr():
        a.lr = float("nan")
        a.step(g, max_norm=limit)

    def bad_betas():
        a.bt = S.betas(0.9, 1.5, 1e-8, 0.0)
        a.step(g, max_norm=limit)

    before = g.clone()
    for call in (bad_lr, bad_betas, lambda: a.step(g, max_norm=0.0), lambda: a.step(g, max_norm=float("nan")),
                 lambda: a.step(g.cpu(), max_norm=limit), lambda: a.step(g[:1].contiguous(), max_norm=limit),
                 lambda: a.step(g.double(), max_norm=limit), lambda: a.step(None, max_norm=limit)):
        with pytest.raises((ValueError, S.ScapeError)):
            call()
        a.lr, a.bt = lr, bt
        assert torch.equal(g, before) and a.t == 0 and a.nonfinite_count() == 0 and (a.grad_norm == 0).all()
    a.step(g, max_norm=limit)
    assert a.nonfinite_count() == 1 and not torch.equal(g[0], before[0]) and torch.equal(g[1], before[1])
    g.copy_(before)
    b.step(g, max_norm=limit)
    for name in ("params", "m", "v", "e"):
        assert torch.equal(getattr(a, name).nan_to_num(9.0), getattr(b, name).nan_to_num(9.0)), name


def test_token_logprobs_leaves_its_workspace(S):
    """The workspace is reserved: two calls at once may share one."""
    ws = scratch(S.token_logprobs_workspace_bytes(5, 40000, 9))
    x, y = torch.randn(5, 40000, device=DEV), torch.arange(5, device=DEV)
    logp, ids = torch.empty(5, device=DEV), torch.empty(5, 9, dtype=torch.int32, device=DEV)
    w = torch.ones(5, device=DEV)
    S.token_logprobs(x, y, logp, ws, top_ids=ids, dlogp=w, dlogits=x)
    assert (ws == 0x5A).all()
