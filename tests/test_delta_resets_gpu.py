"""dg around tokens whose decay is zero: exactly zero there, and neither side's
size reaches the other's rounding."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import delta_grads, rel
from test_delta_gpu import F32, make, ref_args

pytestmark = pytest.mark.gpu

RESETS = [[0], [63], [64], [5, 6, 7], [10, 37, 64, 96, 100, 149], [31, 32, 33, 95, 127, 128], list(range(150))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("at", RESETS, ids=lambda at: "all" if len(at) == 150 else "_".join(map(str, at)))
def test_dg_is_zero_where_the_decay_is(at, h0, dtype):
    """With sizes of dy that alternate by 2^14 from one reset to the next.  A dg
    is a sum of dq_s.q_s - dv_s.v_s over tokens between the same two resets, and
    dq_s and dv_s of a head are each off by F32 of their 2-norm: so dg_t is off
    by at most F32 times the sum of |dq_s| |q_s| + |dv_s| |v_s| over them (a few
    tokens cancel to much less than that)."""
    L = 150
    d, o, dy, dfin = make(1, L, 4, 2, 24, 32, dtype, h0, seed=60)
    for i, t in enumerate(at):
        d["g"][:, t] = [-torch.inf, -200.0, -110.0][i % 3]
        if i % 2 == 0:
            dy[:, t:] *= 2.0 ** -14
        else:
            dy[:, t:] *= 2.0 ** 14
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=None)["dg"]
    torch.cuda.synchronize()
    assert not got[:, at].any()
    a, kw = ref_args(d, o, 32 ** -0.5)
    a[3] = a[3].clamp(min=-1e4)
    a[:2] = [x.repeat_interleave(2, 2) for x in a[:2]]   # a head's own dq
    ref = delta_grads(*a, dy, **kw)
    want = ref["dg"]
    terms = sum(ref[n].norm(dim=-1) * x.double().norm(dim=-1) for n, x in (("dq", a[0]), ("dv", a[2])))
    edge = [0] + at + [L]
    for s, e in zip(edge, edge[1:]):
        if s == e:
            continue
        off, most = (got[:, s:e] - want[:, s:e]).abs().amax(1), F32 * terms[:, s:e].sum(1)
        assert (off <= most).all(), (s, e, off, most)


def test_dg_in_packed_rows_with_resets():
    d, o, dy, dfin = make(1, 200, 4, 2, 24, 32, "f32", True, seed=61, lens=[[70, 1, 64, 65]])
    at = [0, 20, 70, 100, 134, 135, 199]
    d["g"][:, at] = -torch.inf
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)["dg"]
    torch.cuda.synchronize()
    assert not got[:, at].any()
    a, kw = ref_args(d, o, 32 ** -0.5)
    a[3] = a[3].clamp(min=-1e4)
    assert rel(got, delta_grads(*a, dy, **kw, dfin=dfin)["dg"]) <= 4 * F32
