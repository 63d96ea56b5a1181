"""The README's examples as they stand, against a recorder in the place of the
calls that need a GPU."""

import os
import re

import pytest

from sparse_communication_distributed_amd import scape as S

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example(word):
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), flags=re.S)
    found = [b for b in blocks if word in b]
    assert len(found) == 1
    return found[0]


def test_backward_example_adds_up_micro_batches(monkeypatch):
    """Every call that writes a part of the gradient row sets it in the first
    micro-batch and adds to it in the others."""
    tokens, hidden, out = 6, 64, 8
    calls = []
    for name in ("act_alloc", "rmsnorm_pack", "wgrad", "rmsnorm_backward"):
        monkeypatch.setattr(S, name, lambda *a, _n=name, **kw: calls.append((_n, a, kw)) or _n)
    grads = torch.zeros(2, hidden + out * hidden)
    space = dict(tokens=tokens, hidden=hidden, out=out, grads=grads, worker=1, off_g=0, off_w=hidden, dres=None)
    for name in ("x", "gamma", "y", "rstd", "res", "h", "dout", "ws", "dy", "dh", "norm_ws"):
        space[name] = object()
    span = (grads[1].data_ptr(), grads[1].data_ptr() + grads[1].numel() * 4)
    for micro_batch in range(3):
        calls.clear()
        exec(example("rmsnorm_backward"), dict(space, micro_batch=micro_batch))
        writers = [(n, a, kw) for n, a, kw in calls
                   if any(torch.is_tensor(t) and span[0] <= t.data_ptr() < span[1] for t in a)]
        assert [n for n, _, _ in writers] == ["wgrad", "rmsnorm_backward"]
        for n, _, kw in writers:
            assert kw.get("accumulate", False) == (micro_batch > 0), n
