"""What lmc_rotate, lmc_append_rotated, lmc_linear_step and lmc_linear_scan say of
calls at the ends of their ranges (no GPU): nothing is enqueued."""
import numpy as np
import pytest

import test_linear_cpu as C
import workloads as W


@pytest.fixture()
def env(lmc):
    layers = [W.kda(768, 3, 4, 64), W.mla(1152), W.swa(64, 128), W.kda(4, 1, 4, 64)]
    L = lmc.lmc_layout_build(layers, 64, False, 1 << 24)
    buf = np.zeros(4096 + 256, dtype=np.uint8)
    return L, (buf.ctypes.data + 255) // 256 * 256, buf


def test_rotations_of_more_rows_than_a_grid_has_blocks_for(lmc, env):
    """As the header has it: OVERFLOW, and lmc_append's INVALID_ARG where rows are appended."""
    L, base, _ = env
    assert C._rotate(lmc, base, n=1 << 40, out=1 << 60) == lmc.LMC_ERR_OVERFLOW
    assert C._rotate(lmc, base, n=1 << 40, out=1 << 60, xr=517, xh=129) == lmc.LMC_ERR_OVERFLOW
    assert C._append(lmc, L, base, n=1 << 40) == lmc.LMC_ERR_INVALID_ARG
