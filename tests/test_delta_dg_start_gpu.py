"""dg of a row's first tokens where an initial state comes in: what happens
behind them does not reach its rounding."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import delta_grads
from test_delta_gpu import F32, make, ref_args

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,P,N,lens", [(64, 24, 32, None), (50, 130, 64, None), (150, 24, 200, None), (60, 700, 16, None),
                                        (120, 40, 32, [[60, 1, 59]])])
def test_first_tokens(L, P, N, lens, dtype):
    """dy is 2^14 larger from token 40 on, and decays of e^-1 and less a token keep
    that from the first ones.  dg_t = <dh0, h0> - sum_{s<t} (dq_s.q_s - dv_s.v_s),
    each of these off by F32 of the 2-norms it is made of."""
    d, o, dy, _ = make(2, L, 4, 2, P, N, dtype, True, seed=90, lens=None if lens is None else lens * 2, g_max=1.0)
    d["g"] -= 1.0
    dy[:, 40:] *= 2.0 ** 14
    got = ssd.delta_bwd(**d, dy=dy, **o)["dg"]
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, N ** -0.5)
    a[:2] = [x.repeat_interleave(2, 2) for x in a[:2]]
    ref = delta_grads(*a, dy, **kw)
    terms = sum(ref[n].norm(dim=-1) * x.double().norm(dim=-1) for n, x in (("dq", a[0]), ("dv", a[2])))
    h0 = (ref["dinitial_states"].flatten(2).norm(dim=-1) * o["initial_states"].double().flatten(2).norm(dim=-1))[:, None]
    most = F32 * (h0 + terms.cumsum(1))
    for t in range(20):
        assert ((got[:, t] - ref["dg"][:, t]).abs() <= most[:, t]).all(), (t, (got[:, t] - ref["dg"][:, t]).abs(), most[:, t])
