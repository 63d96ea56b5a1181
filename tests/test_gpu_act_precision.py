"""Precision of the weight gradient where a plain sum in fp32 would lose what
the operator promises to keep.  Every expected value is exact: the inputs are
made so that the sums fit 24 bits in the order that the operator takes."""

import numpy as np
import pytest

from oracle import act_oracle as A
from tests.test_gpu_act import DEV, Guarded, exact_inputs, f32, fill_act

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


@pytest.mark.parametrize("rows,n_in,n_out", [(30, 96, 40), (1, 1, 1), (300, 777, 129), (70, 2100, 24), (129, 33, 64),
                                             (5000, 136, 200), (5000, 130, 64), (3, 20001, 5), (700, 3, 1),
                                             (257, 2048, 72), (4100, 32, 8), (128, 1056, 2056)])
def test_wgrad_fp16_columns_of_unlike_size(S, rows, n_in, n_out):
    """Blocks of 32 columns whose scales lie up to 2^180 apart, each block
    uniformly large or small, one all zero: exact in every one of them."""
    q, s, dyn = exact_inputs(rows, n_in, n_out, "fp16", rows + n_in)
    r = np.random.default_rng(n_out)
    base = r.choice(np.array([-107, -60, -31, 0, 40, 73]), s.shape[1])
    base[0], base[-1] = 73, -107
    s = np.where(s == 0, 0, s.astype(np.int64) + base).astype(np.uint8)
    if s.shape[1] > 2:
        s[:, 1], q[:, 32:64] = 0, 0
    gain = np.ldexp(1.0, r.integers(-8, 9, n_in)).astype(np.float32)
    for pad, lead in ((0, 0), (5, 1)):
        dy = Guarded(rows, n_out, torch.float16, pad, lead, dyn)
        need = S.wgrad_workspace_bytes(rows, n_in, n_out, dy.t)
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)
        dw, db = torch.empty(n_out, n_in, device=DEV), torch.empty(n_out, device=DEV)
        S.wgrad(dy.t, fill_act(S, q, s, n_in), dw, ws[:need], gain=torch.from_numpy(gain).to(DEV), dbias=db)
        want, wb = A.wgrad(dyn, A.unpack(q, s, n_in), gain)
        assert (want.astype(np.float32) == want).all()
        got = f32(dw)
        assert (got == want).all(), f"{int((got != want).sum())} of {want.size} differ"
        assert (f32(db) == wb).all()
        assert (ws[need:] == 0xFF).all()


def test_wgrad_fp16_rows_of_unlike_size(S):
    """Within a block rows may lie 2^32 apart and stay exact: the large rows'
    gradient is zero here, so that the small ones are all there is."""
    rows, n_in, n_out = 200, 70, 24
    q, s, dyn = exact_inputs(rows, n_in, n_out, "fp16", 4)
    big = np.arange(rows) % 3 == 0
    base = np.array([60, 120, 30])
    s = np.where(s == 0, 0, base + np.where(big[:, None], 32, s.astype(np.int64) - 126)).astype(np.uint8)
    dyn[big] = 0.0
    dy = Guarded(rows, n_out, torch.float16, 0, 0, dyn)
    ws = torch.empty(S.wgrad_workspace_bytes(rows, n_in, n_out, dy.t), dtype=torch.uint8, device=DEV)
    dw = torch.empty(n_out, n_in, device=DEV)
    S.wgrad(dy.t, fill_act(S, q, s, n_in), dw, ws)
    want, _ = A.wgrad(dyn, A.unpack(q, s, n_in))
    assert (want.astype(np.float32) == want).all() and (f32(dw) == want).all()


@pytest.mark.parametrize("rows,n_in,n_out", [(700, 200, 136), (3000, 136, 200)])
def test_wgrad_fp16_captured_with_other_scales(S, rows, n_in, n_out):
    """A captured call finds the scales of what lies in its buffers when it is
    replayed, in a workspace that other calls have used in between."""
    dt = torch.float16
    first = exact_inputs(rows, n_in, n_out, "fp16", 1)
    a, dy = fill_act(S, first[0], first[1], n_in), torch.from_numpy(first[2]).to(DEV, dt)
    ws = torch.empty(S.wgrad_workspace_bytes(rows, n_in, n_out, dy), dtype=torch.uint8, device=DEV)
    dw, db = torch.empty(n_out, n_in, device=DEV), torch.empty(n_out, device=DEV)
    S.wgrad(dy, a, dw, ws, dbias=db)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.wgrad(dy, a, dw, ws, dbias=db)
    for i, shift in enumerate((0, -90, 70, -40)):
        q, s, dyn = exact_inputs(rows, n_in, n_out, "fp16", 10 + i)
        s = np.where(s == 0, 0, s.astype(np.int64) + shift + 20 * (np.arange(s.shape[1]) % 3)).astype(np.uint8)
        a.codes.copy_(torch.from_numpy(q))
        a.scales.copy_(torch.from_numpy(s))
        dy.copy_(torch.from_numpy(dyn))
        dw.fill_(-1.0)
        db.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        want, wb = A.wgrad(dyn, A.unpack(q, s, n_in))
        assert (want.astype(np.float32) == want).all()
        assert (f32(dw) == want).all() and (f32(db) == wb).all(), i
        ws.fill_(0xFF)
