"""Precision of the weight gradient where a plain sum in fp32 would lose what
the operator promises to keep.  Every expected value is exact: the inputs are
made so that the sums fit 24 bits in the order that the operator takes."""

import numpy as np
import pytest

from oracle import act_oracle as A
from tests.test_gpu_act import DEV, DT, Guarded, f32, fill_act

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def S():
    from sparse_communication_distributed_amd import scape
    scape.lib()
    return scape


@pytest.mark.parametrize("n_in,n_out", [(64, 64), (777, 129), (33, 1531), (1536, 8192)])
def test_wgrad_fp32_small_terms_are_kept(S, n_in, n_out):
    """dy = A (1 + 2^-12 + 2^-23) needs three bf16 terms.  Over 128 rows (too
    few for a second split) and power-of-two inputs the sum is
    128 A c (1 + 2^-12 + 2^-23), 24 bits wide, and every partial sum fits them
    when the small terms are added first.  Added last, 16 rows' third terms
    are 2^-19 beside 128, whose last place is 2^-16: all of them would go."""
    rows = 128
    r = np.random.default_rng(n_in + n_out)
    a_o = np.ldexp(1.0, r.integers(-3, 4, n_out)) * r.choice([-1.0, 1.0], n_out)
    q = np.zeros((rows, A.BLOCK * -(-n_in // A.BLOCK)), dtype=np.int8)
    q[:, :n_in] = np.ldexp(1.0, r.integers(0, 7, n_in)) * r.choice([-1, 1], n_in)
    s = np.full((rows, q.shape[1] // A.BLOCK), 127, dtype=np.uint8)
    dyn = np.tile(a_o * (1 + 2.0 ** -12 + 2.0 ** -23), (rows, 1))
    dy = Guarded(rows, n_out, torch.float32, 1, 1, dyn)
    assert np.array_equal(f32(dy.t).astype(np.float64), dyn)
    ws = torch.empty(S.wgrad_workspace_bytes(rows, n_in, n_out, dy.t), dtype=torch.uint8, device=DEV)
    dw, db = torch.empty(n_out, n_in, device=DEV), torch.empty(n_out, device=DEV)
    S.wgrad(dy.t, fill_act(S, q, s, n_in), dw, ws, dbias=db)
    want = rows * dyn[0][:, None] * q[0, :n_in].astype(np.float64)[None, :]
    assert (want.astype(np.float32) == want).all()
    got, got_b = f32(dw), f32(db)
    assert (got == want).all(), f"{int((got != want).sum())} of {want.size} differ"
    assert (got_b == rows * dyn[0]).all()
