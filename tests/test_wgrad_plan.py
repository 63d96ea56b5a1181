"""The division of the weight gradient's work: sizes that take each tile shape,
with and without splits of the rows.  The GPU tests of the tile shapes run on
these sizes, so a change of the rule that moves one shows here."""

import ctypes
import os

import pytest

from sparse_communication_distributed_amd import scape as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(S.LIB_PATH), reason="libscape.so not built")

# rows, in, out -> splits, tile along out, tile along in, of every type.  The rows fill each ring
# of stages several times and end inside a stage; no tile shape divides in or out.
PLANS = [
    ((587, 1500, 2500), (1, 128, 128)),
    ((1003, 200, 264), (7, 128, 128)),
    ((587, 1500, 2888), (1, 256, 128)),
    ((4099, 264, 3896), (5, 256, 128)),
    ((587, 2900, 2888), (1, 256, 192)),
    ((8191, 264, 5600), (5, 256, 192)),
    ((587, 4090, 2888), (1, 256, 256)),
    ((8191, 2000, 1288), (5, 256, 256)),
]


@pytest.mark.parametrize("size,plan", PLANS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_sizes_take_their_tile_shape(size, plan, dtype):
    assert S.wgrad_splits(*size, dtype) == plan
    rows, n_in, n_out = size
    assert rows % 32 and n_out % plan[1] and n_in % plan[2]


def test_invalid_sizes_have_no_plan():
    m = ctypes.c_int32(-5)
    f = S.lib().scape_wgrad_splits
    for rows, n_in, n_out, dt in ((-1, 8, 8, 1), (1 << 31, 8, 8, 1), (1, 0, 8, 1), (1, 8, (1 << 20) + 1, 1),
                                  (1, 1 << 20, 1 << 20, 1), (1, 8, 8, 3), (1, 8, 8, -1)):
        assert f(rows, n_in, n_out, dt, ctypes.byref(m), None) == -1 and m.value == -5
    assert f(0, 8, 8, 1, None, None) == 1
    with pytest.raises(ValueError):
        S.wgrad_splits(8, 8, 8, torch.float64)
