"""The activation operators at the sizes where their loops turn over: rings of
stages that are filled again, partial tiles, splits, and more rows than the
workgroups of a launch take in one turn."""

import numpy as np
import pytest

from oracle import act_oracle as A
from tests.test_gpu_act import DEV, DT, EPS, HALF, LEAST, U, f32, fill_act, spread, within
from tests.test_wgrad_plan import PLANS

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def S():
    from sparse_communication_distributed_amd import scape
    scape.lib()
    return scape


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def lying(rows, cols, dtype, values, aligned):
    """A [rows][cols] matrix of these values; not aligned: off by one element,
    in rows of odd length."""
    ld, lead = (cols, 0) if aligned else (cols + 1 + cols % 2, 1)
    t = torch.full((rows * ld + lead,), float("nan"), dtype=dtype, device=DEV)[lead:].view(rows, ld)[:, :cols]
    t.copy_(values)
    return t


def whole_checkpoint(S, rows, n_in, seed, powers=False):
    """A checkpoint of whole and half numbers, and its values in binary64."""
    g, nb = gen(seed), -(-n_in // A.BLOCK)
    if powers:
        q = (1 << torch.randint(0, 7, (rows, nb * A.BLOCK), device=DEV, generator=g))
        q = q * (2 * torch.randint(0, 2, q.shape, device=DEV, generator=g) - 1)
    else:
        q = torch.randint(-127, 128, (rows, nb * A.BLOCK), device=DEV, generator=g)
    s = torch.randint(126, 129, (rows, nb), device=DEV, generator=g)
    s = torch.where(torch.rand(rows, nb, device=DEV, generator=g) < 0.1, 0, s)
    q = torch.where((s == 0).repeat_interleave(A.BLOCK, 1), 0, q)
    q[:, n_in:] = 0
    a = S.ActCheckpoint(q.to(torch.int8), s.to(torch.uint8), n_in)
    scale = torch.where(s == 0, 0.0, torch.exp2((s - 127).double()))
    return a, (q.double() * scale.repeat_interleave(A.BLOCK, 1))[:, :n_in].contiguous()


# ----------------------------------------------------------- weight gradient

@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size,plan", PLANS)
def test_wgrad_rings_splits_and_edges(S, size, plan, dt, aligned):
    """Whole numbers whose sums are exact in fp32 in any order, with the bias,
    a gain, and once more added to the result."""
    rows, n_in, n_out = size
    assert S.wgrad_splits(*size, DT[dt]) == plan
    a, x = whole_checkpoint(S, rows, n_in, rows + n_in)
    # |sum| < 2^24 half units, each |x| at most 508 of them
    top = max(1, int(2 ** 24 // (508 * rows)))
    dyv = torch.randint(-top, top + 1, (rows, n_out), device=DEV, generator=gen(n_out)).double()
    dy = lying(rows, n_out, DT[dt], dyv, aligned)
    want, wb = dyv.t().contiguous() @ x, dyv.sum(0)
    ws = torch.full((S.wgrad_workspace_bytes(rows, n_in, n_out, dy),), 0xFF, dtype=torch.uint8, device=DEV)
    dw, db = torch.full((n_out, n_in), -7.0, device=DEV), torch.full((n_out,), -7.0, device=DEV)
    gain = torch.exp2(torch.randint(-3, 4, (n_in,), device=DEV, generator=gen(3)).float())
    S.wgrad(dy, a, dw, ws, gain=gain, dbias=db)
    assert torch.equal(dw.double(), want * gain.double()) and torch.equal(db.double(), wb)
    dw.fill_(2.0)
    S.wgrad(dy, a, dw, ws, dbias=db, accumulate=True)
    # 2 and a sum of at most 2^24 half units
    assert torch.equal(dw.double(), (want + 2).float().double()) and torch.equal(db.double(), 2 * wb)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size,plan", PLANS)
def test_wgrad_every_bit_and_every_row(S, size, plan, dt):
    """One nonzero gradient a column of dy, of all the type's bits, over rows
    that reach each stage, and codes that are powers of two: products and sums
    are exact, and a row, column or term out of place shows."""
    rows, n_in, n_out = size
    a, x = whole_checkpoint(S, rows, n_in, n_in + n_out, powers=True)
    bits = {"fp32": 24, "bf16": 8, "fp16": 11}[dt]
    r = np.random.default_rng(rows)
    at = np.resize(np.concatenate([[rows - 1, 0], r.permutation(rows)]), n_out)  # the last row and the first among them
    v = (r.integers(1 << (bits - 1), 1 << bits, n_out) | 1) * r.choice([-1.0, 1.0], n_out)
    dyv = torch.zeros(rows, n_out, dtype=torch.float64, device=DEV)
    at_t, v_t = torch.from_numpy(at).to(DEV), torch.from_numpy(v).to(DEV)
    dyv[at_t, torch.arange(n_out, device=DEV)] = v_t
    dy = lying(rows, n_out, DT[dt], dyv, True)
    assert torch.equal(dy.double(), dyv)
    ws = torch.empty(S.wgrad_workspace_bytes(rows, n_in, n_out, dy), dtype=torch.uint8, device=DEV)
    dw, db = torch.empty(n_out, n_in, device=DEV), torch.empty(n_out, device=DEV)
    S.wgrad(dy, a, dw, ws, dbias=db)
    assert torch.equal(dw.double(), v_t[:, None] * x[at_t]) and torch.equal(db.double(), v_t)


@pytest.mark.parametrize("rows,n_in,n_out", [(300, 260, 130), (5000, 136, 200)])
def test_wgrad_fp16_values_within_one_term(S, rows, n_in, n_out):
    """fp16 is multiplied once: exact products, one sum of `rows` of them."""
    q, s = A.pack(spread(rows, n_in, 21).astype(np.float32))
    a, x8 = fill_act(S, q, s, n_in), A.unpack(q, s, n_in)
    dy = torch.from_numpy(spread(rows, n_out, 22)).to(DEV, torch.float16)
    dyn = f32(dy).astype(np.float64)
    want, wb = A.wgrad(dyn, x8)
    ws = torch.empty(S.wgrad_workspace_bytes(rows, n_in, n_out, dy), dtype=torch.uint8, device=DEV)
    dw, db = torch.empty(n_out, n_in, device=DEV), torch.empty(n_out, device=DEV)
    S.wgrad(dy, a, dw, ws, dbias=db)
    # each partial sum is off by at most a unit in the last place of a magnitude below the whole's
    within(dw, want, 2 * U * (rows + 8) * (np.abs(dyn).T @ np.abs(x8)), "dw")
    within(db, wb, U * (rows + 8) * np.abs(dyn).sum(axis=0), "dbias")


# ---------------------------------------------------- more rows than a turn

FORWARD_TURNS = [(262144 + 4097, 40), (65536 + 77, 520), (65536 + 1030, 1030), (65536 + 9, 2056), (65536 + 5, 16392)]


@pytest.mark.parametrize("rows,cols", FORWARD_TURNS)
def test_rmsnorm_rows_past_the_grid(S, rows, cols):
    """Workgroups that take a second row: every row equals the same row in a
    call on a part of the rows, whose own results the oracle pins."""
    x = torch.randn(rows, cols, device=DEV, generator=gen(1), dtype=torch.bfloat16)
    x[::7] *= 3.0
    w = torch.randn(cols, device=DEV, generator=gen(2))
    y, a, rstd = torch.empty_like(x), S.act_alloc(rows, cols, DEV), torch.empty(rows, device=DEV)
    S.rmsnorm_pack(x, w, EPS, y, xhat=a, rstd=rstd)
    part = 16384
    y2, r2 = torch.empty(part, cols, dtype=x.dtype, device=DEV), torch.empty(part, device=DEV)
    for i in range(0, rows, part):
        m = min(part, rows - i)
        b = S.act_alloc(m, cols, DEV)
        S.rmsnorm_pack(x[i:i + m], w, EPS, y2[:m], xhat=b, rstd=r2[:m])
        assert torch.equal(y[i:i + m], y2[:m]) and torch.equal(rstd[i:i + m], r2[:m])
        assert torch.equal(a.codes[i:i + m], b.codes) and torch.equal(a.scales[i:i + m], b.scales)
    for i in (0, 65535, 65536, rows - 3):  # and some rows against the oracle
        hs = f32(x[i:i + 3])
        rs = rstd[i:i + 3].cpu().numpy()
        assert (np.abs(rs - A.norm_rstd(hs, EPS)) <= A.norm_rstd(hs, EPS) * U * (1 + 1e-6)).all()
        q, s = A.pack(hs * rs[:, None])
        assert np.array_equal(a.codes[i:i + 3].cpu().numpy(), q) and np.array_equal(a.scales[i:i + 3].cpu().numpy(), s)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,cols", [(5000, 264), (4101, 505), (2500, 1280), (2500, 1030), (2500, 4096), (1030, 8192),
                                       (700, 16384), (600, 16392)])
def test_rmsnorm_backward_turns(S, rows, cols, dt):
    """More rows than workgroups: the next row is loaded while one is
    computed, and a workgroup's part of dweight is a sum of several."""
    t = DT[dt]
    g = gen(rows + cols)
    rnd = lambda *sh: torch.randn(*sh, device=DEV, generator=g)  # noqa: E731
    a, x8 = S.act_alloc(rows, cols, DEV), torch.empty(rows, cols, device=DEV)
    S.act_pack(rnd(rows, cols), a)
    S.act_unpack(a, x8)
    x8 = x8.double()
    rstd, w = torch.exp(rnd(rows)), rnd(cols)
    dy, dres = (rnd(rows, cols) * torch.exp(rnd(rows, 1))).to(t), rnd(rows, cols).to(t)
    ws = torch.empty(S.rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    dh, dw = torch.empty_like(dy), torch.empty(cols, device=DEV)
    S.rmsnorm_backward(dy, a, rstd, w, dh, dw, ws, dres=dres)
    d, r64, rs = dy.double(), dres.double(), rstd.double()[:, None]
    gy = d * w.double()
    want = rs * (gy - x8 * (gy * x8).mean(1, keepdim=True)) + r64
    # the bound of the smaller sizes' test: the roundings of each formula, counted
    gv, mean_abs = gy.abs(), (gy * x8).abs().mean(1, keepdim=True)
    depth = cols / 64 + 24
    mag = rs * (gv + x8.abs() * mean_abs) + r64.abs()
    tol = U * (rs * (5 * gv + x8.abs() * mean_abs * (depth + 5)) + 2 * r64.abs()) * 1.01
    tol = tol + HALF[t] * torch.minimum(want.abs() + tol, mag * 1.01) + 2 * LEAST[t]
    assert ((dh.double() - want).abs() <= tol).all()
    size = (d * x8).abs().sum(0)
    assert ((dw.double() - (d * x8).sum(0)).abs() <= U * (rows + 16) * size * 1.01 + 1e-45).all()
    # the same with dh in dy's place
    p, dw2 = dy.clone(), torch.empty_like(dw)
    S.rmsnorm_backward(p, a, rstd, w, p, dw2, ws, dres=dres)
    assert torch.equal(p, dh) and torch.equal(dw2, dw)


@pytest.mark.parametrize("cols", [264, 520, 1280, 5000, 17000])
def test_rmsnorm_backward_one_tensor_as_both_gradients(S, cols):
    rows = 300
    g = gen(6)
    x, dy = (torch.randn(rows, cols, device=DEV, dtype=torch.bfloat16, generator=g) for _ in range(2))
    w = torch.randn(cols, device=DEV, generator=g)
    a, rstd = S.act_alloc(rows, cols, DEV), torch.empty(rows, device=DEV)
    S.rmsnorm_pack(x, w, EPS, xhat=a, rstd=rstd)
    ws = torch.empty(S.rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    one, two, dw1, dw2 = torch.empty_like(dy), torch.empty_like(dy), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    S.rmsnorm_backward(dy, a, rstd, w, one, dw1, ws, dres=dy)
    S.rmsnorm_backward(dy, a, rstd, w, two, dw2, ws, dres=dy.clone())
    assert torch.equal(one, two) and torch.equal(dw1, dw2)
    S.rmsnorm_backward(dy, a, rstd, w, dy, dw1, ws, dres=dy)  # and the result in its place
    assert torch.equal(dy, two) and torch.equal(dw1, dw2)


@pytest.mark.parametrize("cols", [16392, 40000])
def test_rmsnorm_backward_long_rows_past_the_grid(S, cols):
    """More long rows than the workgroups of a launch (65536)."""
    rows = 65536 + 3
    if cols > 20000:
        rows = 300  # the partial sums' walk alone
    dy = torch.randn(rows, cols, device=DEV, generator=gen(7), dtype=torch.bfloat16)
    a = S.act_alloc(rows, cols, DEV)
    S.act_pack(dy, a)
    rstd, w = torch.ones(rows, device=DEV), torch.randn(cols, device=DEV, generator=gen(8))
    ws = torch.empty(S.rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    dh, dw = torch.empty_like(dy), torch.empty(cols, device=DEV)
    S.rmsnorm_backward(dy, a, rstd, w, dh, dw, ws)
    last = slice(rows - 4, rows)
    b = S.ActCheckpoint(a.codes[last], a.scales[last], cols)
    dh2 = torch.empty(4, cols, dtype=dy.dtype, device=DEV)
    S.rmsnorm_backward(dy[last], b, rstd[last], w, dh2, None, ws)
    assert torch.equal(dh[last], dh2)
    assert torch.isfinite(dh[:: max(1, rows // 512)]).all()
    want, size = (torch.zeros(cols, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, rows, 4096):
        m = min(4096, rows - i)
        x8 = torch.empty(m, cols, device=DEV)
        S.act_unpack(S.ActCheckpoint(a.codes[i:i + m], a.scales[i:i + m], cols), x8)
        prod = dy[i:i + m].double() * x8.double()
        want += prod.sum(0)
        size += prod.abs().sum(0)
    # 256 parts of these rows, then 64 groups of 4 parts
    assert ((dw.double() - want).abs() <= U * (rows // 256 + 1 + 4 + 64) * size * 1.01).all()
