"""Refusals and sizes of the embedding, the log probabilities and the clipping
that need no GPU: a refused call returns before anything reaches the device."""

import ctypes
import os

import pytest

from sparse_communication_distributed_amd import scape as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(S.LIB_PATH), reason="libscape.so not built")

FAKE = 0x10000  # non-null, never dereferenced by a refused call
INVALID, SHAPE, WORKSPACE = 1, 2, 3
BF16, FP16 = 1, 2
NAN, INF = float("nan"), float("inf")


def mat(ld=64, dtype=BF16, data=FAKE):
    return S.Matrix(data, ld, dtype)


def ids(bits=64, data=FAKE):
    return S.Ids(data, bits)


NONE, NO_IDS = S.Matrix(None, 0, 0), S.Ids(None, 0)


def call(fn, defaults, **kw):
    d = dict(defaults)
    assert set(kw) <= set(d)
    d.update(kw)
    return fn(*d.values(), None)


EMBED = dict(tokens=4, vocab=9, positions=0, cols=64, ids=ids(), table=mat(), scale=1.0, pos=NO_IDS, pos_table=NONE,
             out=mat(data=2 * FAKE))


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 26) + 1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=1 << 31), SHAPE),
    (dict(cols=0), SHAPE), (dict(cols=(1 << 20) + 1), SHAPE), (dict(ids=NO_IDS), INVALID),
    (dict(ids=ids(16)), INVALID), (dict(ids=ids(64, FAKE + 4)), INVALID), (dict(ids=ids(32, FAKE + 2)), INVALID),
    (dict(table=NONE), INVALID), (dict(table=mat(63)), SHAPE), (dict(table=mat(dtype=3)), INVALID),
    (dict(table=mat(data=FAKE + 1)), INVALID), (dict(out=NONE), INVALID), (dict(out=mat(63)), SHAPE),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(pos_table=mat()), SHAPE),  # no positions
    (dict(pos_table=mat(), positions=1 << 31), SHAPE), (dict(pos_table=mat(), positions=5), INVALID),  # no pos
    (dict(pos_table=mat(dtype=0), positions=5, pos=ids()), INVALID),
    (dict(pos_table=mat(63), positions=5, pos=ids()), SHAPE),
])
def test_embed_refuses(kw, status):
    assert call(S.lib().scape_embed, EMBED, **kw) == status
    assert S.lib().scape_last_error()


BACK = dict(tokens=4, vocab=9, cols=64, ids=ids(), dy=mat(), scale=1.0, dtable=FAKE, accumulate=0, workspace=FAKE,
            nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(cols=0), SHAPE), (dict(ids=NO_IDS), INVALID),
    (dict(ids=ids(8)), INVALID), (dict(dy=NONE), INVALID), (dict(dy=mat(10)), SHAPE), (dict(dy=mat(dtype=9)), INVALID),
    (dict(scale=INF), INVALID), (dict(dtable=None), INVALID), (dict(dtable=FAKE + 2), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace=FAKE + 128), INVALID), (dict(nbytes=0), WORKSPACE),
])
def test_embed_backward_refuses(kw, status):
    assert call(S.lib().scape_embed_backward, BACK, **kw) == status


LOGP = dict(rows=4, vocab=64, logits=mat(), scale=1.0, targets=ids(), logp=FAKE, stats=None, entropy=None, top=0,
            top_logp=None, top_ids=None, dlogp=None, dentropy=None, dlogits=NONE, workspace=FAKE, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 20) + 1), SHAPE), (dict(top=-1), SHAPE),
    (dict(top=65, top_ids=FAKE), SHAPE), (dict(top=33, vocab=32, top_ids=FAKE), SHAPE),
    (dict(logits=NONE), INVALID), (dict(logits=mat(63)), SHAPE), (dict(logits=mat(dtype=5)), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(scale=2.0 ** 101), INVALID), (dict(scale=2.0 ** -101), INVALID),
    (dict(targets=NO_IDS), INVALID), (dict(targets=ids(7)), INVALID), (dict(logp=FAKE + 1), INVALID),
    (dict(stats=FAKE + 2), INVALID), (dict(entropy=FAKE + 3), INVALID), (dict(logp=None), INVALID),  # no output
    (dict(top=4), INVALID), (dict(top_ids=FAKE), INVALID), (dict(top_logp=FAKE), INVALID),
    (dict(top=4, top_ids=FAKE + 2), INVALID), (dict(dlogp=FAKE), INVALID), (dict(dentropy=FAKE), INVALID),
    (dict(dlogits=mat()), INVALID),  # no weight
    (dict(dlogits=mat(dtype=FP16), dlogp=FAKE), INVALID), (dict(dlogits=mat(66), dlogp=FAKE), INVALID),
    (dict(dlogits=mat(60, data=2 * FAKE), dlogp=FAKE), SHAPE), (dict(dlogits=mat(), dlogp=FAKE + 1), INVALID),
    (dict(dlogits=mat(), dlogp=FAKE, targets=NO_IDS, logp=None), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace=FAKE + 64), INVALID), (dict(nbytes=0), WORKSPACE),
])
def test_token_logprobs_refuses(kw, status):
    assert call(S.lib().scape_token_logprobs, LOGP, **kw) == status


LBACK = dict(rows=4, vocab=64, logits=mat(), scale=1.0, targets=ids(), stats=FAKE, entropy=FAKE, dlogp=FAKE,
             dentropy=FAKE, dlogits=mat(data=2 * FAKE))


@pytest.mark.parametrize("kw,status", [
    (dict(rows=1 << 31), SHAPE), (dict(logits=NONE), INVALID), (dict(scale=0.0), INVALID),
    (dict(targets=NO_IDS), INVALID), (dict(stats=None), INVALID), (dict(stats=FAKE + 2), INVALID),
    (dict(entropy=None), INVALID), (dict(entropy=FAKE + 2), INVALID), (dict(dlogp=None, dentropy=None), INVALID),
    (dict(dlogits=NONE), INVALID), (dict(dlogits=mat(dtype=0, data=2 * FAKE)), INVALID),
    (dict(dlogits=mat(65)), INVALID), (dict(dlogits=mat(4, data=2 * FAKE)), SHAPE), (dict(dentropy=FAKE + 2), INVALID),
])
def test_token_logprobs_backward_refuses(kw, status):
    assert call(S.lib().scape_token_logprobs_backward, LBACK, **kw) == status


def grads(*items):
    return (S.Grad * len(items))(*items)


def grad(data=FAKE, out=None, count=10, dtype=BF16, out_dtype=0):
    return S.Grad(data, out, count, dtype, out_dtype)


@pytest.mark.parametrize("items,groups,status", [
    ([grad()] * 3, 2, SHAPE), ([grad()], 0, SHAPE), ([grad(count=-1)], 1, SHAPE),
    ([grad(count=(1 << 46) + 1)], 1, SHAPE), ([grad(count=1 << 45)] * 3, 1, SHAPE), ([grad(data=None)], 1, INVALID),
    ([grad(), grad(dtype=3)], 1, INVALID), ([grad(data=FAKE + 1)], 1, INVALID),
])
def test_grad_list_refuses(items, groups, status):
    L, g = S.lib(), grads(*items)
    assert L.scape_grad_workspace_bytes(len(g), g, groups) == 0
    assert L.scape_grad_norm(len(g), g, groups, 1.0, FAKE, FAKE, 1 << 40, None) == status
    assert L.scape_grad_clip(len(g), g, groups, 1.0, 1.0, FAKE, FAKE, 1 << 40, None) == status


@pytest.mark.parametrize("count,groups", [((1 << 20) + 1, 1), ((1 << 21), 1 << 21), (0, (1 << 20) + 1)])
def test_grad_list_refuses_more_than_a_launch_holds(count, groups):
    L = S.lib()
    g = (S.Grad * max(count, 1))()  # counts of 0: refused by the list's length alone
    assert L.scape_grad_workspace_bytes(count, g, groups) == 0
    assert L.scape_grad_norm(count, g, groups, 1.0, FAKE, FAKE, 1 << 40, None) == SHAPE
    assert L.scape_grad_clip(count, g, groups, 1.0, 1.0, FAKE, FAKE, 1 << 40, None) == SHAPE


@pytest.mark.parametrize("item", [
    grad(out=2 * FAKE, out_dtype=FP16), grad(out=2 * FAKE, out_dtype=7), grad(out=2 * FAKE + 2, out_dtype=0),
    grad(out=FAKE, out_dtype=0),  # fp32 in the place of bf16
])
def test_grad_clip_refuses_places(item):
    g = grads(item)
    assert S.lib().scape_grad_clip(1, g, 1, 1.0, 1.0, FAKE, FAKE, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(max_norm=0.0), INVALID),
    (dict(max_norm=-1.0), INVALID), (dict(max_norm=NAN), INVALID), (dict(norm=None), INVALID),
    (dict(norm=FAKE + 2), INVALID), (dict(workspace=None), INVALID), (dict(workspace=FAKE + 8), INVALID),
    (dict(nbytes=0), WORKSPACE),
])
def test_grad_clip_refuses(kw, status):
    d = dict(count=1, grads=grads(grad()), groups=1, scale=1.0, max_norm=1.0, norm=FAKE, workspace=FAKE,
             nbytes=1 << 40)
    assert call(S.lib().scape_grad_clip, d, **kw) == status
    d.pop("max_norm")
    if "max_norm" not in kw:
        assert call(S.lib().scape_grad_norm, d, **kw) == status


def test_sizes():
    assert S.token_logprobs_max_top() == 64
    for rows, vocab, top in ((-1, 5, 0), (1 << 31, 5, 0), (1, 0, 0), (1, 5, 6), (1, 100, 65), (1, 5, -1)):
        assert S.token_logprobs_workspace_bytes(rows, vocab, top) == 0
    for tokens, cols in ((-1, 5), ((1 << 26) + 1, 5), (5, 0)):
        assert S.embed_workspace_bytes(tokens, cols) == 0
    for n in (0, 1, 16384):
        assert S.embed_workspace_bytes(n, 2048) % 256 == 0 and S.embed_workspace_bytes(n, 2048) > 0
        assert S.token_logprobs_workspace_bytes(n, 32000, 20) % 256 == 0
        assert S.token_logprobs_workspace_bytes(n, 32000, 20) > 0
    L = S.lib()
    assert L.scape_grad_workspace_bytes(0, None, 1) > 0
    # no more partial sums than a long list needs
    assert L.scape_grad_workspace_bytes(2, grads(grad(count=1 << 40), grad(count=1 << 40)), 2) < 1 << 18


def test_binding_refuses():
    """Host tensors, wrong types and shapes are named before any address is taken."""
    host = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="table must be a device tensor"):
        S.embed(torch.zeros(4, dtype=torch.int64), host, host)
    with pytest.raises(ValueError, match="dy must be a device tensor"):
        S.embed_backward(torch.zeros(4, dtype=torch.int64), host, host, host)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        S.token_logprobs(host, torch.zeros(4, dtype=torch.int64), None, host)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        S.token_logprobs_backward(host, None, None, host)
    with pytest.raises(ValueError, match="logits must be a tensor"):
        S.token_logprobs(None, None, None, None)
    with pytest.raises(ValueError, match=r"grads\[0\] must be a device tensor"):
        S.GradList([host])
    with pytest.raises(ValueError, match="grads is empty"):
        S.GradList([])
    with pytest.raises(ValueError, match="equal parts"):
        S.GradList([host] * 3, groups=2)
    with pytest.raises(ValueError, match=r"out must have 1 tensors"):
        S.GradList([host], out=[])
    with pytest.raises(ValueError, match="must be a GradList"):
        S.grad_norm([host], host, host)
    with pytest.raises(ValueError, match="must be a GradList"):
        S.clip_grads(host, 1.0, host, host)
