"""How much workspace the norm's backward asks for (no call here reaches a kernel)."""
import ctypes

import pytest

import mamba_ssd_chunked_03_b200 as ssd


def need(rows, cols, dtype=ssd.SSD_BF16):
    a = ssd.NormBwdArgs(rows, cols, dtype, 1e-5)
    return int(ssd.lib.ssd_layer_norm_bwd_workspace_size(ctypes.byref(a)))


def up(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("dtype", [ssd.SSD_BF16, ssd.SSD_F32])
@pytest.mark.parametrize("rows,cols", [(1, 4), (1, 1), (7, 5120), (3, 20000), (1000, 64), (50, 4096), (50, 4097)])
def test_few_rows_take_no_more_than_their_sums(rows, cols, dtype):
    assert need(rows, cols, dtype) == up(8 * rows * cols) + (up(12 * rows) if cols > 4096 else 0)


@pytest.mark.parametrize("rows,cols", [(1 << 30, 4), ((1 << 31) - 1, 1), (100_000_000, 64), (16384, 2560)])
def test_many_rows_take_what_the_grid_does(rows, cols):
    assert need(rows, cols) == up(8 * 148 * 16384)


def test_wide_rows():
    assert need(16384, 100_000) == up(8 * 444 * 100_000) + up(12 * 16384)
    assert need((1 << 31) - 1, (1 << 31) - 1) == up(8 * 444 * ((1 << 31) - 1)) + up(12 * ((1 << 31) - 1))
