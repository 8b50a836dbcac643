"""Layer norm where its calls are easiest to get wrong.  Bounds as in test_norm."""
import ctypes

import pytest

import exact_flow_recurrence_gb300 as efla
from test_norm import BF, F32, _check


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,D", [(40000, 64), (20000, 1024), (4500, 4096), (1600, 8192), (1500, 16384), (5000, 333)])
def test_many_rows_a_group(rows, D, dtype):
    """Every group of warps takes ten rows and more: the ring's stages (six at most, one in the widest fp32
    backward) are filled again and change phase."""
    _check(rows, D, dtype, F32, True, seed=D)
    _check(rows, D, dtype, BF, False, pad=8, seed=D + 1)


def test_stats_must_lie_on_8_bytes():
    """A row's mean and rstd are read and written as one pair.  Host checks: nothing is launched (no GPU needed)."""
    lib = efla.load_library()
    p = [0x7f0000000000 + i * 0x10000000 for i in range(8)]
    for dtype in (efla.BF16, efla.F32):
        s = ctypes.byref(efla.NormShape(rows=4, D=64, x_stride=64, y_stride=64, dtype=dtype, weight_dtype=efla.F32, eps=1e-5))
        assert lib.efla_norm_fwd(s, p[0], p[1], None, p[2], p[3] + 4, None) == 3
        assert b"stats" in lib.efla_last_error()
        assert lib.efla_norm_bwd(s, p[0], p[1], p[2], p[3] + 4, p[4], p[5], p[6], p[7], 1 << 24, None) == 3
        assert b"stats" in lib.efla_last_error()
        # (a refused workspace proves that stats + 8 passed: it is checked later)
        assert lib.efla_norm_bwd(s, p[0], p[1], p[2], p[3] + 8, p[4], p[5], p[6], None, 0, None) == 4
