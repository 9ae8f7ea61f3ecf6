"""The decode step's grid: what does not fit is refused on the host, for every
width of the state, before anything is launched."""
import ctypes

import pytest

import mamba_ssd_chunked_03_b200 as ssd
from test_delta_cpu import UNS, step_args


@pytest.mark.parametrize("dstate", [4, 16, 20, 32, 36, 64, 68, 128, 132, 256])
@pytest.mark.parametrize("batch,nheads,headdim", [(1 << 29, 4, 1), (1 << 25, 4, 256), (1 << 17, 4, 65536), (1 << 31, 1, 16),
                                                  (1 << 40, 1 << 22, 65536)])
def test_step_grid(batch, nheads, headdim, dstate):
    """16 rows of a state or fewer for each CTA: 2^31 of them are too many."""
    a = step_args(batch=batch, nheads=nheads, headdim=headdim, dstate=dstate, ngroups=1)
    assert ssd.lib.ssd_delta_step(ctypes.byref(a), None) == UNS
