"""The embedding, the log probabilities and the clipping as a program uses
them: a model's whole training step into the optimizer, other streams, two at
once, captured passes, refusals of the binding."""

import numpy as np
import pytest

from oracle import ends_oracle as E

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"


@pytest.fixture(scope="module")
def S():
    from sparse_communication_distributed_amd import scape
    scape.lib()
    return scape


def scratch(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


class Model:
    """Embedding (with positions), RMS norm, output product, loss: one worker's
    step into its row of the gradients, [table | positions | norm | head]."""

    EPS = 1e-5

    def __init__(self, S, tokens, vocab, positions, hidden, dtype, seed):
        self.S, self.tokens, self.vocab, self.positions, self.hidden = S, tokens, vocab, positions, hidden
        self.dtype = dtype
        sizes = [vocab * hidden, positions * hidden, hidden, vocab * hidden]
        self.at = np.concatenate([[0], np.cumsum(sizes)]).tolist()
        self.n = self.at[-1] + (-self.at[-1]) % 4
        g = torch.Generator(DEV).manual_seed(seed)
        self.w = torch.zeros(self.n, device=DEV)
        self.w[:self.at[4]] = 0.3 * torch.randn(self.at[4], device=DEV, generator=g)
        self.w[self.at[2]:self.at[3]] = 1.0
        new = lambda *s, t=dtype: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
        self.h, self.y, self.dy, self.dh = (new(tokens, hidden) for _ in range(4))
        self.logits = new(tokens, vocab)
        self.logp, self.rstd = new(tokens, t=torch.float32), new(tokens, t=torch.float32)
        self.xhat = S.act_alloc(tokens, hidden, DEV)
        self.pos = torch.arange(tokens, device=DEV) % positions
        self.ids = torch.zeros(tokens, dtype=torch.int64, device=DEV)
        self.targets = torch.zeros(tokens, dtype=torch.int64, device=DEV)
        self.weight = new(tokens, t=torch.float32)
        self.row = new(self.n, t=torch.float32).zero_()
        self.ws = [scratch(n) for n in (S.embed_workspace_bytes(tokens, hidden),
                                        S.token_logprobs_workspace_bytes(tokens, vocab),
                                        S.wgrad_workspace_bytes(tokens, hidden, vocab),
                                        S.rmsnorm_workspace_bytes(tokens, hidden))]
        self.norm = new(1, t=torch.float32)
        self.list = S.GradList([self.row])
        self.clip_ws = scratch(S.grad_workspace_bytes(self.list))

    def draw(self, seed):
        r = np.random.default_rng(seed)
        ids = r.integers(0, self.vocab, self.tokens)
        ids[r.random(self.tokens) < 0.1] = -100
        y = r.integers(0, self.vocab, self.tokens)
        y[r.random(self.tokens) < 0.1] = -100
        self.ids.copy_(torch.from_numpy(ids))
        self.targets.copy_(torch.from_numpy(y))
        self.weight.fill_(-1.0 / self.tokens)

    def part(self, i, buf=None):
        return (self.w if buf is None else buf)[self.at[i]:self.at[i + 1]]

    def table(self, i, buf=None):
        return self.part(i, buf).view(-1, self.hidden)

    def step(self, max_norm=None, micro=0):
        """Forward and backward; logits in place become their gradient."""
        S = self.S
        S.embed(self.ids, self.table(0), self.h, scale=2.0, pos=self.pos, pos_table=self.table(1))
        S.rmsnorm_pack(self.h, self.part(2), self.EPS, self.y, xhat=self.xhat, rstd=self.rstd)
        head = self.table(3).to(self.dtype)
        torch.mm(self.y, head.t(), out=self.logits)
        S.token_logprobs(self.logits, self.targets, self.logp, self.ws[1], dlogp=self.weight, dlogits=self.logits)
        S.wgrad(self.logits, self.xhat, self.part(3, self.row), self.ws[2], gain=self.part(2), accumulate=micro > 0)
        torch.mm(self.logits, head, out=self.dy)
        S.rmsnorm_backward(self.dy, self.xhat, self.rstd, self.part(2), self.dh, self.part(2, self.row), self.ws[3],
                           accumulate=micro > 0)
        S.embed_backward(self.ids, self.dh, self.table(0, self.row), self.ws[0], scale=2.0, accumulate=micro > 0)
        S.embed_backward(self.pos, self.dh, self.table(1, self.row), self.ws[0], accumulate=micro > 0)
        if max_norm is not None:
            S.clip_grads(self.list, max_norm, self.norm, self.clip_ws)

    def results(self):
        return [t.clone() for t in (self.logp, self.logits, self.row, self.norm)]


def reference(m):
    """Loss and gradient row of the same model in 64 bits, by torch's own
    derivatives of the forward formulas (on the host)."""
    w = m.w.double().cpu().requires_grad_()
    part = lambda i: w[m.at[i]:m.at[i + 1]]  # noqa: E731
    ids, pos, y = m.ids.cpu(), m.pos.cpu(), m.targets.cpu()
    h = torch.where((ids >= 0)[:, None], 2.0 * part(0).view(-1, m.hidden)[ids.clamp(min=0)], 0.0)
    h = h + part(1).view(-1, m.hidden)[pos]
    xh = h / torch.sqrt((h * h).mean(1, keepdim=True) + m.EPS)
    x = (xh * part(2)) @ part(3).view(-1, m.hidden).t()
    lp = x - torch.logsumexp(x, 1, keepdim=True)
    logp = torch.where(y >= 0, lp.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
    loss = -logp.sum() / m.tokens
    loss.backward()
    return logp.detach().numpy(), w.grad.numpy()


def test_training_step_against_derivatives(S):
    """The row of gradients that the whole chain writes, fp32 throughout, is
    the derivative of the loss; the only coarse rounding is the 8-bit
    checkpoint of the normalised rows (half a quantum of 1/63.5 of a block's
    largest value at most, about 1/250 of its spread here)."""
    m = Model(S, 300, 61, 20, 64, torch.float32, 1)
    m.draw(2)
    m.step()
    logp, want = reference(m)
    assert np.abs(m.logp.cpu().numpy() - logp).max() < 1e-4  # |logits| of some tens, 64 products: 64 * 2^-24 * 30
    got = m.row.double().cpu().numpy()
    for i, name in enumerate(("table", "positions", "norm", "head")):
        a, b = got[m.at[i]:m.at[i + 1]], want[m.at[i]:m.at[i + 1]]
        # every entry of the checkpoint is off by half a quantum at most: a block's largest value over 127, a share
        # of at most 1/127 * 32^(1/2) of the block's 2-norm; the gradients are linear in it
        assert np.linalg.norm(a - b) <= 32 ** 0.5 / 127 * np.linalg.norm(b), name
    assert (got[m.at[4]:] == 0).all()


def test_micro_batches_add_up(S):
    m = Model(S, 200, 40, 10, 32, torch.bfloat16, 3)
    parts = []
    for i in range(2):
        m.draw(10 + i)
        m.row.fill_(7.0)
        m.step()
        parts.append(m.row[:m.at[4]].double())
    m.draw(10)
    m.step()
    m.draw(11)
    m.step(micro=1)
    both = parts[0] + parts[1]
    # sums of the same numbers in another order: 200 and 400 terms of 32 bits
    bound = 400 * 2.0 ** -24 * (m.row[:m.at[4]].double().abs().max() + both.abs().max())
    assert (m.row[:m.at[4]].double() - both).abs().max() <= bound


def test_clipped_rows_step_like_the_oracle(S):
    """Two workers' rows, clipped by their own norms, through the optimizer:
    the step equals the step oracle on the rows the clipping left."""
    from oracle import scape_oracle as O
    K, P = 2, 4
    m = Model(S, 64, 33, 8, 32, torch.bfloat16, 4)
    k = m.n // P // 10
    opt = S.ScapeOptimizer(m.w.clone(), P, K, k)
    ora = O.OracleOptimizer(m.w.cpu().numpy(), P, K, k, O.Hyper.make(0.9, 0.95, 1e-8, 0.0, 1e-3))
    grads = torch.zeros(K, m.n, device=DEV)
    for t in range(1, 4):
        for i in range(K):
            m.draw(100 * t + i)
            m.step()
            grads[i].copy_(m.row * (1.0 + 3 * i))
        before = grads.double().cpu().numpy()
        norms = [E.grad_norm([r]) for r in before]
        limit = float(np.float32(0.5 * (norms[0] + norms[1])))
        opt.step(grads, max_norm=limit)
        assert np.allclose(opt.grad_norm.cpu().numpy(), norms, rtol=2.0 ** -23, atol=0)
        after = grads.cpu().numpy()
        for i in range(K):
            f = E.clip_factor(norms[i], limit)
            assert (f < 1) == (i == 1)
            assert (np.abs(after[i] - before[i] * f) <= np.abs(before[i] * f) * 2.0 ** -24 * (1 + 1e-6)).all()
        ora.step(after)
        torch.cuda.synchronize()
        for name, want in (("params", ora.gather("w")), ("m", ora.gather("m")), ("e", ora.gather("e"))):
            assert np.array_equal(getattr(opt, name).cpu().numpy().view(np.uint32), want.view(np.uint32)), (t, name)
        m.w.copy_(opt.params)


def test_other_stream_and_repeat(S):
    m = Model(S, 3000, 700, 100, 48, torch.bfloat16, 5)
    m.draw(6)
    m.step(max_norm=0.01)
    want = m.results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        m.row.fill_(5.0)
        m.row[m.at[4]:] = 0.0
        m.logits.fill_(1.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.step(max_norm=0.01)
        side.synchronize()
        for a, b in zip(m.results(), want):
            assert torch.equal(a, b)
    # the stream as an argument, the current one another
    out, ref = torch.empty_like(m.h), torch.empty_like(m.h)
    S.embed(m.ids, m.table(0), ref)
    torch.cuda.synchronize()
    S.embed(m.ids, m.table(0), out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)


def test_two_streams_at_once(S):
    ms = [Model(S, 2500 + 17 * i, 900, 64, 40, t, 7 + i) for i, t in enumerate((torch.bfloat16, torch.float16))]
    want = []
    for i, m in enumerate(ms):
        m.draw(20 + i)
        m.step(max_norm=0.02)
        want.append(m.results())
        m.row.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    for _ in range(4):
        for m, s in zip(ms, streams):
            with torch.cuda.stream(s):
                m.step(max_norm=0.02)
    torch.cuda.synchronize()
    for m, w in zip(ms, want):
        for a, b in zip(m.results(), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,vocab", [(600, 130), (17000, 50)])
def test_captured_and_replayed(S, tokens, vocab):
    """Replays with new inputs, and the program's own passes between them: two
    graphs that share every buffer and workspace."""
    m = Model(S, tokens, vocab, 30, 32, torch.bfloat16, 9)
    m.draw(1)
    m.step(max_norm=0.05)
    torch.cuda.synchronize()
    graphs = []
    for limit in (0.05, 1e6):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.step(max_norm=limit)
        graphs.append((g, limit))
    for i in range(4):
        for g, limit in graphs:
            m.draw(30 + i)
            m.row.fill_(3.0)
            m.row[m.at[4]:] = 0.0
            g.replay()
            torch.cuda.synchronize()
            got = m.results()
            m.row.fill_(4.0)
            m.row[m.at[4]:] = 0.0
            m.step(max_norm=limit)
            torch.cuda.synchronize()
            for a, b in zip(got, m.results()):
                assert torch.equal(a, b), (i, limit)


def test_serving_forms_captured(S):
    """Single tokens: embedding, probabilities and alternatives of one row, as
    replayed between samples."""
    vocab, hidden = 32000, 128
    table = torch.randn(vocab, hidden, device=DEV)
    ids, out = torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty(1, hidden, dtype=torch.bfloat16, device=DEV)
    logits = torch.empty(1, vocab, dtype=torch.bfloat16, device=DEV)
    logp, h = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    top, lp = torch.empty(1, 20, dtype=torch.int32, device=DEV), torch.empty(1, 20, device=DEV)
    ws = scratch(S.token_logprobs_workspace_bytes(1, vocab, 20))

    def run():
        S.embed(ids, table, out)
        S.token_logprobs(logits, ids, logp, ws, entropy=h, top_logp=lp, top_ids=top, scale=1.25)

    logits.normal_()
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(4):
        ids.fill_(i * 7001)
        logits.copy_(3 * torch.randn(1, vocab, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, logp, h, top, lp)]
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, logp, h, top, lp)))
        want, _ = E.top(logits.double().cpu().numpy(), 20, 1.25)
        assert np.array_equal(top.cpu().numpy(), want)


def test_binding_refuses(S):
    d = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    i64 = torch.int64
    table, ids, out, ws = d(9, 8), d(4, t=i64), d(4, 8), scratch(1 << 16)
    for match, call in (
        ("ids must be int32 or int64", lambda: S.embed(d(4), table, out)),
        ("ids must be contiguous with 4", lambda: S.embed(d(5, t=i64), table, out)),
        ("ids must be contiguous with 4", lambda: S.embed(d(8, t=i64)[::2], table, out)),
        ("ids must be a tensor on device", lambda: S.embed(torch.zeros(4, dtype=i64), table, out)),
        ("out must have shape", lambda: S.embed(ids, table, d(4, 9))),
        ("out must have consecutive", lambda: S.embed(ids, table, d(8, 4).t())),
        ("pos needs pos_table", lambda: S.embed(ids, table, out, pos=ids)),
        ("pos_table must have shape", lambda: S.embed(ids, table, out, pos=ids, pos_table=d(3, 7))),
        ("SCAPE_EINVAL: pos_table must have table's dtype",
         lambda: S.embed(ids, table, out, pos=ids, pos_table=d(3, 8, t=torch.bfloat16))),
        ("table must be float32, bfloat16", lambda: S.embed(ids, d(9, 8, t=torch.float64), out)),
        ("dtable must have 8 columns", lambda: S.embed_backward(ids, out, d(9, 7), ws)),
        ("dtable must be a float32", lambda: S.embed_backward(ids, out, d(9, 8, t=torch.bfloat16), ws)),
        ("dtable must be contiguous", lambda: S.embed_backward(ids, out, d(9, 9)[:, :8], ws)),
        ("workspace is too small", lambda: S.embed_backward(ids, out, table, scratch(256))),
        ("workspace must be 256-byte", lambda: S.embed_backward(ids, out, table, ws[8:])),
        ("workspace must be a tensor", lambda: S.embed_backward(ids, out, table, None)),
        ("logp must be contiguous with 4", lambda: S.token_logprobs(d(4, 9), ids, d(3), ws)),
        ("SCAPE_EINVAL: targets is null", lambda: S.token_logprobs(d(4, 9), None, d(4), ws)),
        ("SCAPE_EINVAL: every output is null", lambda: S.token_logprobs(d(4, 9), ids, None, ws)),
        ("top_ids must be an int32", lambda: S.token_logprobs(d(4, 9), ids, None, ws, top_ids=d(4, 3))),
        ("top_logp must have shape", lambda: S.token_logprobs(d(4, 9), ids, None, ws, top_logp=d(4, 2),
                                                              top_ids=d(4, 3, t=torch.int32))),
        ("workspace is too small|SCAPE_ESHAPE", lambda: S.token_logprobs(d(4, 9), ids, None, ws, top_logp=d(4, 10))),
        ("stats must be contiguous with 8", lambda: S.token_logprobs(d(4, 9), ids, None, ws, stats=d(4))),
        ("dlogits must have shape", lambda: S.token_logprobs(d(4, 9), ids, None, ws, dlogp=d(4), dlogits=d(4, 8))),
        ("SCAPE_EINVAL: dlogits must have logits' dtype",
         lambda: S.token_logprobs(d(4, 9), ids, None, ws, dlogp=d(4), dlogits=d(4, 9, t=torch.float16))),
        ("SCAPE_EINVAL: stats is null", lambda: S.token_logprobs_backward(d(4, 9), ids, None, d(4, 9), dlogp=d(4))),
        ("SCAPE_EINVAL: entropy is null",
         lambda: S.token_logprobs_backward(d(4, 9), ids, d(4, 2), d(4, 9), dentropy=d(4))),
        (r"grads\[1\] must be contiguous", lambda: S.GradList([table, d(8, 4).t()])),
        (r"grads\[0\] must be float32", lambda: S.GradList([ids])),
        (r"out\[0\] must have 72 elements", lambda: S.GradList([table], out=[d(71)])),
        (r"out\[0\] must be torch.bfloat16 or float32",
         lambda: S.GradList([d(4, t=torch.bfloat16)], out=[d(4, t=torch.float16)])),
        ("max_norm must be positive", lambda: S.clip_grads(S.GradList([table]), 0.0, d(1), ws)),
        ("norm must be contiguous with 1", lambda: S.clip_grads(S.GradList([table]), 1.0, d(2), ws)),
        ("workspace is too small", lambda: S.grad_norm(S.GradList([table]), d(1), scratch(0))),
    ):
        with pytest.raises((ValueError, S.ScapeError), match=match):
            call()


def test_grad_lists_that_overlap(S):
    buf, n, ws = torch.randn(100, device=DEV), torch.zeros(1, device=DEV), scratch(1 << 16)
    a, b, c = buf[:40], buf[40:80], buf[30:50]
    other = torch.empty(100, device=DEV)
    for gl in (S.GradList([a, a]), S.GradList([a, b, c]), S.GradList([a], out=[buf[1:41]]),
               S.GradList([a, b], out=[other[:40], other[39:79]]), S.GradList([a, b], out=[buf[40:80], other[:40]]),
               S.GradList([buf, other[:4]], out=[other, buf[20:24]])):
        with pytest.raises(ValueError, match="overlaps another tensor"):
            S.clip_grads(gl, 1.0, n, ws)
        S.grad_norm(gl, n, ws)  # reads only
        want = sum(float((g.double() ** 2).sum()) for g in gl.grads) ** 0.5
        if torch.isfinite(other).all():
            assert abs(n.item() - want) <= 1e-6 * want
    for gl in (S.GradList([a, b]), S.GradList([a, a], out=[other[:40], other[40:80]]), S.GradList([a], out=[a]),
               S.GradList([buf[:0], a, buf[:0]])):
        S.clip_grads(gl, 1.0, n, ws)
