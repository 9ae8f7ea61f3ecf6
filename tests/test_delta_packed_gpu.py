"""Packed rows of the delta rule's backward: gradients handed in for ids that do
not occur, and the check of the ids."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from test_delta_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_absent_ids_do_not_matter(dtype):
    """ids 1 and 3 do not occur: what dfinal_states holds for them reaches nothing."""
    d, o, dy, dfin = make(1, 100, 4, 2, 24, 32, dtype, True, seed=80, lens=[[20, 50, 30]], ids=[4, 0, 2])
    want = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    dfin[1], dfin[3] = float("nan"), float("inf")
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    assert all(torch.equal(got[n], want[n]) and torch.isfinite(got[n]).all() for n in got)


def test_backward_checks_the_ids_when_asked():
    d, o, dy, _ = make(1, 90, 2, 1, 16, 16, "bf16", seed=81, lens=[[30, 30, 30]])
    want = ssd.delta_bwd(**d, dy=dy, **o)
    got = ssd.delta_bwd(**d, dy=dy, **o, check_seq=True)
    assert all(torch.equal(got[n], want[n]) for n in got if got[n] is not None)
    bad = o["seq_idx"].clone()
    bad[0, 60:] = 0                            # an id that comes back
    with pytest.raises(ssd.SSDError):
        ssd.delta_bwd(**d, dy=dy, seq_idx=bad, num_seqs=3, check_seq=True)
    bad[0, 60:] = 3                            # an id out of range
    with pytest.raises(ssd.SSDError):
        ssd.delta_bwd(**d, dy=dy, seq_idx=bad, num_seqs=3, check_seq=True)
