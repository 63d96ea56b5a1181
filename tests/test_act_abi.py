"""Refusals and sizes of the activation operators' C ABI and binding that
need no GPU: a refused call returns before anything reaches the device."""

import ctypes
import os

import pytest

from sparse_communication_distributed_amd import scape as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(S.LIB_PATH), reason="libscape.so not built")

FAKE = 0x10000  # non-null, never dereferenced by a refused call
INVALID, SHAPE, WORKSPACE = 1, 2, 3
BF16 = 1


def mat(ld=64, dtype=BF16, data=FAKE):
    return S.Matrix(data, ld, dtype)


NONE = S.Matrix(None, 0, 0)
ACT = S.ActView(FAKE, FAKE)
NO_ACT = S.ActView(None, None)


def test_sizes():
    assert S.lib().scape_act_block() == S.ACT_BLOCK == 32
    assert S.act_bytes(8, 64) == 512 + 256
    assert S.act_bytes(1, 33) == 256 + 256
    assert S.act_bytes(0, 5) > 0
    for rows, cols in ((-1, 5), (1 << 31, 5), (1, 0), (1, (1 << 20) + 1)):
        assert S.act_bytes(rows, cols) == 0 and S.rmsnorm_workspace_bytes(rows, cols) == 0
        assert S.wgrad_workspace_bytes(rows, cols, 8) == 0 and S.wgrad_workspace_bytes(rows, 8, cols) == 0
    assert S.wgrad_workspace_bytes(4, 1 << 20, 1 << 20) == 0
    assert S.rmsnorm_workspace_bytes(4096, 1280) % 256 == 0
    # the workspace for any dy covers each type's, aligned or not
    L, most = S.lib(), S.wgrad_workspace_bytes(999, 100, 72)
    sizes = [L.scape_wgrad_workspace_bytes(999, 100, 72, m)
             for m in (mat(72), mat(73), mat(72, data=FAKE + 2), mat(72, 2), mat(72, 0))]
    assert sizes[0] < sizes[1] == sizes[2] <= sizes[4] == most
    assert L.scape_wgrad_workspace_bytes(999, 100, 72, mat(73, 2)) <= most
    v = S.ActView()
    assert S.lib().scape_act_slot(8, 64, FAKE, ctypes.byref(v)) == 0
    assert v.codes == FAKE and v.scales == FAKE + 512
    assert S.lib().scape_act_slot(8, 64, None, ctypes.byref(v)) == INVALID


@pytest.mark.parametrize("args,status", [
    ((-1, 64, mat(), ACT), SHAPE),
    ((4, 0, mat(), ACT), SHAPE),
    ((4, 64, mat(63), ACT), SHAPE),
    ((1 << 30, 64, mat(1 << 20), ACT), SHAPE),  # rows * ld past 2^46
    ((4, 64, mat(dtype=7), ACT), INVALID),
    ((4, 64, mat(data=FAKE + 1), ACT), INVALID),
    ((4, 64, NONE, ACT), INVALID),
    ((4, 64, mat(), NO_ACT), INVALID),
    ((4, 64, mat(), S.ActView(FAKE, None)), INVALID),
    ((4, 64, mat(), S.ActView(FAKE + 8, FAKE)), INVALID),
])
def test_pack_and_unpack_refuse(args, status):
    L = S.lib()
    rows, cols, m, a = args
    assert L.scape_act_pack(rows, cols, m, a, None) == status
    assert L.scape_act_unpack(rows, cols, a, None, m, None) == status
    assert L.scape_last_error()


def norm_args(**kw):
    d = dict(rows=4, cols=64, x=mat(), residual=NONE, weight=FAKE, eps=1e-5, h=NONE, y=mat(data=2 * FAKE), xhat=NO_ACT,
             rstd=None)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(rows=1 << 31), SHAPE),
    (dict(cols=(1 << 20) + 1), SHAPE),
    (dict(x=NONE), INVALID),
    (dict(y=NONE), INVALID),  # neither y nor xhat
    (dict(weight=None), INVALID),
    (dict(weight=FAKE + 2), INVALID),
    (dict(rstd=FAKE + 2), INVALID),
    (dict(eps=0.0), INVALID),
    (dict(eps=-1e-5), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(residual=mat(dtype=2)), INVALID),
    (dict(y=mat(dtype=0, data=2 * FAKE)), INVALID),
    (dict(h=mat(ld=10)), SHAPE),
    (dict(h=mat(data=2 * FAKE)), INVALID),  # h and y in one place
    (dict(h=mat(ld=80)), INVALID),  # in x's place with another ld
    (dict(xhat=S.ActView(None, FAKE)), INVALID),
])
def test_rmsnorm_pack_refuses(kw, status):
    assert S.lib().scape_rmsnorm_pack(*norm_args(**kw)) == status


def back_args(**kw):
    d = dict(rows=4, cols=64, dy=mat(), xhat=ACT, rstd=FAKE, weight=FAKE, dres=NONE, dh=mat(data=2 * FAKE),
             dweight=FAKE, accumulate=0, workspace=FAKE, nbytes=1 << 30)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE),
    (dict(dy=NONE), INVALID),
    (dict(xhat=NO_ACT), INVALID),
    (dict(rstd=None), INVALID),
    (dict(weight=None), INVALID),
    (dict(dh=NONE, dweight=None), INVALID),
    (dict(dweight=FAKE + 1), INVALID),
    (dict(dres=mat(dtype=0)), INVALID),
    (dict(dh=mat(dtype=2)), INVALID),
    (dict(dh=mat(ld=72)), INVALID),  # in dy's place with another ld
    (dict(dres=mat(ld=63)), SHAPE),
    (dict(workspace=None), INVALID),
    (dict(workspace=FAKE + 16), INVALID),
    (dict(nbytes=S.rmsnorm_workspace_bytes(4, 64) - 1), WORKSPACE),
])
def test_rmsnorm_backward_refuses(kw, status):
    assert S.lib().scape_rmsnorm_backward(*back_args(**kw)) == status


def wgrad_args(**kw):
    d = dict(rows=4, n_in=64, n_out=64, dy=mat(), x=ACT, gain=None, dw=FAKE, dbias=None, accumulate=0,
             workspace=FAKE, nbytes=1 << 30)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE),
    (dict(n_in=0), SHAPE),
    (dict(n_out=0), SHAPE),
    (dict(n_in=1 << 20, n_out=1 << 20, dy=mat(1 << 20)), SHAPE),
    (dict(dy=mat(32)), SHAPE),
    (dict(dy=NONE), INVALID),
    (dict(x=NO_ACT), INVALID),
    (dict(dw=None), INVALID),
    (dict(dw=FAKE + 2), INVALID),
    (dict(gain=FAKE + 2), INVALID),
    (dict(dbias=FAKE + 1), INVALID),
    (dict(workspace=None), INVALID),
    (dict(workspace=FAKE + 128), INVALID),
    (dict(nbytes=S.lib().scape_wgrad_workspace_bytes(4, 64, 64, mat()) - 1), WORKSPACE),
    (dict(dy=mat(dtype=0), nbytes=S.lib().scape_wgrad_workspace_bytes(4, 64, 64, mat())), WORKSPACE),
])
def test_wgrad_refuses(kw, status):
    assert S.lib().scape_wgrad(*wgrad_args(**kw)) == status


def test_binding_refuses_host_tensors():
    x, vec = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(ValueError):
        S.ActCheckpoint(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        S.act_pack(x, None)
    with pytest.raises(ValueError):
        S.rmsnorm_pack(x, vec, 1e-5, y=x)
    with pytest.raises(ValueError):
        S.rmsnorm_backward(x, None, vec, vec, x, vec, vec)
    with pytest.raises(ValueError):
        S.act_alloc(4, 64, "cpu")
    with pytest.raises(S.ScapeError):
        S.act_alloc(4, 0, "cpu")


def test_binding_refuses_what_is_not_a_tensor():
    """A missing or foreign argument is named, before anything is called."""
    x, vec = torch.zeros(4, 64), torch.zeros(64)
    for bad, name in ((lambda: S.act_pack(None, None), "x"), (lambda: S.act_unpack(None, x), "a"),
                      (lambda: S.rmsnorm_pack(None, vec, 1e-5, y=x), "x"),
                      (lambda: S.rmsnorm_backward(None, None, vec, vec, x, vec, vec), "dy"),
                      (lambda: S.wgrad(None, None, x, vec), "dy"), (lambda: S.wgrad([1.0], None, x, vec), "dy"),
                      (lambda: S.wgrad_workspace_bytes(4, 64, 64, 3.0), "dy"),
                      (lambda: S._workspace(None, 256, 0), "workspace"), (lambda: S._matrix(2.0, "y", 4, 64, 0), "y"),
                      (lambda: S._vector([0.0] * 64, "weight", 64, 0), "weight"),
                      (lambda: S.ActCheckpoint(None, None, 64), "codes")):
        with pytest.raises(ValueError, match=name):
            bad()
