"""Pointers that are no boundary of their elements are refused before anything is
launched: an access through one would fault."""
import ctypes

import pytest

import mamba_ssd_chunked_03_b200 as ssd
from test_delta_cpu import FAKE, INV, bwd_args, delta_args, norm_args, step_args


def with_workspace(a, size):
    n = getattr(ssd.lib, size)(ctypes.byref(a))
    assert n > 0
    a.workspace, a.workspace_bytes = 1 << 24, n
    return a


@pytest.mark.parametrize("dtype", [ssd.SSD_BF16, ssd.SSD_F32])
@pytest.mark.parametrize("name", ["q", "k", "v", "y", "g", "beta", "initial_states", "final_states", "seq_idx"])
def test_delta_fwd(name, dtype):
    off = 1 if dtype == ssd.SSD_BF16 and name in "qkvy" else 2
    a = with_workspace(delta_args(dtype=dtype, num_seqs=3, **{name: FAKE + off}), "ssd_delta_fwd_workspace_size")
    assert ssd.lib.ssd_delta_fwd(ctypes.byref(a), None) == INV


@pytest.mark.parametrize("dtype", [ssd.SSD_BF16, ssd.SSD_F32])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "initial_states", "seq_idx", "dy", "dq", "dk", "dv", "dg",
                                  "dbeta", "dfinal_states", "dinitial_states"])
def test_delta_bwd(name, dtype):
    off = 1 if dtype == ssd.SSD_BF16 and name in ("q", "k", "v", "dy", "dq", "dk", "dv") else 2
    a = bwd_args(dtype=dtype, num_seqs=3, **{name: FAKE + off})
    assert ssd.lib.ssd_delta_bwd(ctypes.byref(with_workspace(a, "ssd_delta_bwd_workspace_size")), None) == INV


@pytest.mark.parametrize("dtype", [ssd.SSD_BF16, ssd.SSD_F32])
@pytest.mark.parametrize("name", ["v", "y", "g", "beta"])
def test_delta_step(name, dtype):
    off = 1 if dtype == ssd.SSD_BF16 and name in "vy" else 2
    assert ssd.lib.ssd_delta_step(ctypes.byref(step_args(dtype=dtype, **{name: FAKE + off})), None) == INV


@pytest.mark.parametrize("name", ["weight", "bias"])
def test_layer_norm(name):
    assert ssd.lib.ssd_layer_norm(ctypes.byref(norm_args(**{name: FAKE + 2})), None) == INV


@pytest.mark.parametrize("name", ["weight", "bias", "dweight", "dbias"])
def test_layer_norm_bwd(name):
    a = with_workspace(norm_args(ssd.NormBwdArgs, **{name: FAKE + 2}), "ssd_layer_norm_bwd_workspace_size")
    assert ssd.lib.ssd_layer_norm_bwd(ctypes.byref(a), None) == INV
