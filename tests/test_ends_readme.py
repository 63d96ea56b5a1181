"""The README's example of the step's ends, against a recorder in the place of
the calls that need a GPU."""

import pytest

from sparse_communication_distributed_amd import scape as S
from tests.test_readme import example

torch = pytest.importorskip("torch")


def test_ends_example_writes_the_worker_s_part(monkeypatch):
    vocab, hidden, n = 7, 4, 40
    calls = []
    for name in ("embed", "token_logprobs", "embed_backward"):
        monkeypatch.setattr(S, name, lambda *a, _n=name, **kw: calls.append((_n, a, kw)))

    class Opt:
        def step(self, grads, max_norm=None):
            calls.append(("step", (grads,), {"max_norm": max_norm}))

    grads = torch.zeros(3, n)
    space = dict(S=S, opt=Opt(), vocab=vocab, hidden=hidden, grads=grads, worker=2)
    for name in ("ids", "table", "h", "pos", "pos_table", "logits", "targets", "logp", "logp_ws", "weight", "dh",
                 "embed_ws"):
        space[name] = object()
    for micro_batch in range(2):
        calls.clear()
        exec(example("embed_backward"), dict(space, micro_batch=micro_batch))
        assert [c[0] for c in calls] == ["embed", "token_logprobs", "embed_backward", "step"]
        _, args, kw = calls[2]
        assert args[2].shape == (vocab, hidden) and args[2].data_ptr() == grads[2].data_ptr()
        assert kw["accumulate"] == (micro_batch > 0)
        assert calls[3][1][0] is grads and calls[3][2]["max_norm"] == 1.0
        assert calls[1][2]["dlogits"] is space["logits"]
