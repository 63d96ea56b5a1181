"""Lists of gradients keep the memory that they are lists of.  Host tensors
stand for the device's."""

import pytest

from sparse_communication_distributed_amd import scape as S

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("with_out", [False, True])
def test_memory_of_a_list_is_not_reused(monkeypatch, with_out):
    """A tensor given other memory: nothing new lies at its old address, which
    the list reads and writes."""
    def check(self, t, name):
        self.device = 0
        return S._dtype(t.dtype, name)
    monkeypatch.setattr(S.GradList, "_check", check)
    g, o = torch.ones(5000), torch.zeros(5000)
    gl = S.GradList([g], out=[o] if with_out else None)
    old = {g.data_ptr(), o.data_ptr()} if with_out else {g.data_ptr()}
    held = []
    for t in (g, o) if with_out else (g,):
        t.data = torch.zeros(1)
    for n in (5000, 5000, 4999, 100) * 8:
        held.append(torch.zeros(n))
    assert not old & {t.data_ptr() for t in held}
    assert gl.items[0].data in old
