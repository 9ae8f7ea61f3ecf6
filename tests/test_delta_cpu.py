"""Refusals and layouts of the delta rule's and the norm's entry points.  CPU
only: no call here reaches a kernel launch."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from test_abi import _c_layout

FAKE = 1 << 20  # never dereferenced: every case below is rejected on the host
INV, UNS, WS = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_ERR_WORKSPACE


def delta_args(a=None, **kw):
    a = a or ssd.DeltaArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups = 2, 100, 4, 64, 128, 2
    a.dtype, a.scale = ssd.SSD_BF16, 0.1
    a.q = a.k = a.v = a.g = a.beta = a.y = FAKE
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def bwd_args(**kw):
    a = ssd.DeltaBwdArgs()
    delta_args(a.fwd)
    a.dy = a.dq = a.dk = a.dv = a.dg = a.dbeta = FAKE
    for k, v in kw.items():
        setattr(a if hasattr(a, k) else a.fwd, k, v)
    return a


SIZES = [("batch", 0, INV), ("seqlen", -1, INV), ("nheads", 0, INV), ("headdim", 0, INV), ("dstate", 0, INV),
         ("ngroups", 3, INV), ("dtype", 7, INV), ("flags", 4, INV), ("dstate", 257, UNS), ("headdim", 65537, UNS),
         ("batch", 1 << 30, UNS), ("q", None, INV), ("k", None, INV), ("v", None, INV), ("g", None, INV),
         ("beta", None, INV)]


@pytest.mark.parametrize("field,value,status", SIZES + [("y", None, INV)])
def test_delta_fwd_refuses(field, value, status):
    assert ssd.lib.ssd_delta_fwd(ctypes.byref(delta_args(**{field: value})), None) == status


@pytest.mark.parametrize("field,value,status", SIZES + [(n, None, INV) for n in ("dy", "dq", "dk", "dv", "dg", "dbeta")])
def test_delta_bwd_refuses(field, value, status):
    assert ssd.lib.ssd_delta_bwd(ctypes.byref(bwd_args(**{field: value})), None) == status


@pytest.mark.parametrize("entry,size,make", [
    ("ssd_delta_fwd", "ssd_delta_fwd_workspace_size", delta_args),
    ("ssd_delta_bwd", "ssd_delta_bwd_workspace_size", bwd_args)])
def test_delta_workspace_is_checked(entry, size, make):
    call, need_of = getattr(ssd.lib, entry), getattr(ssd.lib, size)
    assert call(None, None) == INV and need_of(None) == 0
    a = make()
    need = need_of(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    assert call(ctypes.byref(a), None) == WS
    a.workspace, a.workspace_bytes = 1 << 24, need - 1
    assert call(ctypes.byref(a), None) == WS
    a.workspace, a.workspace_bytes = (1 << 24) + 16, need
    assert call(ctypes.byref(a), None) == INV
    b = make(seq_idx=FAKE, num_seqs=0)
    assert call(ctypes.byref(b), None) == INV and need_of(ctypes.byref(b)) == 0
    b = make(seq_idx=FAKE, num_seqs=5)
    assert need_of(ctypes.byref(b)) > need


def step_args(**kw):
    a = ssd.DeltaStepArgs()
    a.batch, a.nheads, a.headdim, a.dstate, a.ngroups, a.dtype, a.scale = 2, 4, 64, 128, 2, ssd.SSD_BF16, 0.1
    a.q = a.k = a.v = a.g = a.beta = a.state = a.y = FAKE
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("field,value,status", [
    ("batch", 0, INV), ("nheads", -4, INV), ("headdim", 0, INV), ("dstate", 0, INV), ("ngroups", 3, INV),
    ("dtype", 2, INV), ("dstate", 130, UNS), ("dstate", 260, UNS), ("headdim", 65537, UNS), ("batch", 1 << 29, UNS),
    ("q", None, INV), ("state", None, INV), ("y", None, INV), ("state", FAKE + 4, INV), ("k", FAKE + 2, INV)])
def test_delta_step_refuses(field, value, status):
    assert ssd.lib.ssd_delta_step(ctypes.byref(step_args(**{field: value})), None) == status
    assert ssd.lib.ssd_delta_step(None, None) == INV


def norm_args(cls=ssd.NormArgs, **kw):
    a = cls()
    a.rows, a.cols, a.dtype, a.eps = 8, 64, ssd.SSD_BF16, 1e-5
    a.x = FAKE
    for n in ("out", "dout", "dx"):
        if hasattr(a, n):
            setattr(a, n, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


NORM = [("rows", 0, INV), ("cols", 0, INV), ("cols", -1, INV), ("dtype", 3, INV), ("eps", -1.0, INV),
        ("eps", float("nan"), INV), ("rows", 1 << 31, UNS), ("x", None, INV), ("x", FAKE + 1, INV)]


@pytest.mark.parametrize("field,value,status", NORM + [("out", None, INV), ("z", FAKE + 1, INV)])
def test_layer_norm_refuses(field, value, status):
    assert ssd.lib.ssd_layer_norm(ctypes.byref(norm_args(**{field: value})), None) == status
    assert ssd.lib.ssd_layer_norm(None, None) == INV


@pytest.mark.parametrize("field,value,status", NORM + [("dout", None, INV), ("dx", None, INV), ("z", FAKE, INV),
                                                       ("dz", FAKE, INV)])
def test_layer_norm_bwd_refuses(field, value, status):
    assert ssd.lib.ssd_layer_norm_bwd(ctypes.byref(norm_args(ssd.NormBwdArgs, **{field: value})), None) == status
    assert ssd.lib.ssd_layer_norm_bwd(None, None) == INV


def test_layer_norm_bwd_workspace_is_checked():
    a = norm_args(ssd.NormBwdArgs)
    need = ssd.lib.ssd_layer_norm_bwd_workspace_size(ctypes.byref(a))
    assert need > 0 and ssd.lib.ssd_layer_norm_bwd_workspace_size(None) == 0
    assert ssd.lib.ssd_layer_norm_bwd(ctypes.byref(a), None) == WS
    a.workspace, a.workspace_bytes = 1 << 24, need - 1
    assert ssd.lib.ssd_layer_norm_bwd(ctypes.byref(a), None) == WS
    a.workspace, a.workspace_bytes = (1 << 24) + 8, need
    assert ssd.lib.ssd_layer_norm_bwd(ctypes.byref(a), None) == INV


@pytest.mark.parametrize("cls,struct", [
    (ssd.DeltaArgs, "ssd_delta_args"), (ssd.DeltaBwdArgs, "ssd_delta_bwd_args"), (ssd.DeltaStepArgs, "ssd_delta_step_args"),
    (ssd.NormArgs, "ssd_norm_args"), (ssd.NormBwdArgs, "ssd_norm_bwd_args")])
def test_struct_layouts_match_the_header(cls, struct):
    fields = [n for n, _ in cls._fields_]
    want = _c_layout(fields, struct)
    got = [getattr(cls, n).offset for n in fields] + [ctypes.sizeof(cls)]
    assert list(want) == got


def tensors(b=1, L=8, H=4, G=2, P=16, N=32, dtype=torch.bfloat16):
    return dict(q=torch.zeros(b, L, G, N, dtype=dtype), k=torch.zeros(b, L, G, N, dtype=dtype),
                v=torch.zeros(b, L, H, P, dtype=dtype), g=torch.zeros(b, L, H), beta=torch.zeros(b, L, H))


@pytest.mark.parametrize("name,change,error", [
    ("q", lambda t: t, ValueError),                                   # CPU tensors
    ("q", lambda t: t.float(), TypeError), ("v", lambda t: t.half(), TypeError),
    ("g", lambda t: t.bfloat16(), TypeError), ("beta", lambda t: t[:, 1:], ValueError),
    ("k", lambda t: t[..., 1:], ValueError), ("v", lambda t: t[0], ValueError)])
def test_binding_refuses(name, change, error):
    d = tensors()
    d[name] = change(d[name])
    with pytest.raises(error):
        ssd.delta_fwd(**d)
    with pytest.raises(error):
        ssd.delta_bwd(**d, dy=torch.zeros_like(d["v"]))


def test_binding_refuses_other_tensors():
    d = tensors()
    with pytest.raises(ValueError):
        ssd.delta_fwd(**d, initial_states=torch.zeros(1, 4, 16, 31))
    with pytest.raises(ValueError):
        ssd.delta_fwd(**d, seq_idx=torch.zeros(1, 8, dtype=torch.int64), num_seqs=1)
    with pytest.raises(ValueError):
        ssd.delta_bwd(**d, dy=torch.zeros(1, 8, 4, 15, dtype=torch.bfloat16))
    s = {n: t[:, 0] for n, t in d.items()}
    with pytest.raises(ValueError):
        ssd.delta_step(**s, state=torch.zeros(1, 4, 16, 31))
    with pytest.raises(TypeError):
        ssd.delta_step(**s, state=torch.zeros(1, 4, 16, 32, dtype=torch.float64))
    x = torch.zeros(3, 8)
    for kw in (dict(weight=torch.zeros(7)), dict(bias=torch.zeros(8, dtype=torch.float64)), dict(z=torch.zeros(3, 7)),
               dict()):
        with pytest.raises(ValueError):
            ssd.layer_norm(x, **kw)
    with pytest.raises(TypeError):
        ssd.layer_norm(x.half())
    with pytest.raises(ValueError):
        ssd.layer_norm_bwd(x, None, None, x[:2])
