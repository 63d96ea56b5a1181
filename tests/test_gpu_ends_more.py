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
