"""dg of tokens that decay nearly everything: exp(g) is 1e-4 to 1e-9, and so is dg
against what their neighbours' gradients are made of.  It is held to its own
size, not to theirs."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import delta, delta_grads, rel
from test_delta_gpu import F32, make, ref_args

pytestmark = pytest.mark.gpu


def most_off(d, o, dfin, dy, t, N):
    """2 F32 exp(g_t) |G| |S| of each head: S the state before token t, G the gradient of that state as it enters t undecayed."""
    ids = [0] * d["v"].shape[1] if o["seq_idx"] is None else o["seq_idx"][0].tolist()
    t0, t1 = ids.index(ids[t]), len(ids) - ids[::-1].index(ids[t])
    part = lambda a, b: [d[n][:, a:b] for n in ("q", "k", "v", "g", "beta")]
    S = delta(*part(t0, t), N ** -0.5, o["initial_states"] if t0 == 0 else None)[1]
    rest = part(t, t1)
    rest[3] = rest[3].clone()
    rest[3][:, 0] = 0
    G = delta_grads(*rest, dy[:, t:t1], N ** -0.5, S, dfin=dfin[ids[t]][None])["dinitial_states"]
    return (2 * F32 * d["g"][0, t].double().exp() * G[0].flatten(1).norm(dim=1) * S[0].flatten(1).norm(dim=1)).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("every", [1, 2, 5, 31, 33, 70])
@pytest.mark.parametrize("L,N,lens", [(64, 64, None), (150, 128, None), (97, 200, None), (90, 17, [[33, 1, 56]])])
def test_deep_decays(L, N, lens, every, h0, dtype):
    """All that passes a token carries its decay, and a sum of a few hundred such
    terms is off by F32 of the 2-norm over the tokens of one depth (twice it:
    they cancel by up to that much).  One token by itself may cancel by any
    amount: dg_t = exp(g_t) <G, S>, of a state and a gradient that are each off by
    F32 of their 2-norms."""
    d, o, dy, dfin = make(1, L, 6, 3, 24, N, dtype, h0, seed=95, lens=lens, g_max=0.2)
    deep = torch.arange(L) % every == every - 1
    if not deep.any():
        deep[L // 2] = True
    for h, g in enumerate((-9.0, -12.0, -15.0, -18.0, -20.0, -10.0)):
        d["g"][:, deep, h] = g
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)["dg"]
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, N ** -0.5)
    want = delta_grads(*a, dy, **kw, dfin=dfin)["dg"]
    one = most_off(d, o, dfin, dy, int(deep.nonzero()[0]), N) if deep.sum() == 1 else None
    for h in range(6):
        x, r = got[:, deep, h], want[:, deep, h]
        if one is None:
            assert r.abs().max() < 1e-2 and rel(x, r) <= 2 * F32, (h, rel(x, r))
        else:
            assert (x - r).abs().item() <= one[h], (h, x, r, one[h])
    if not deep.all():
        assert rel(got[:, ~deep], want[:, ~deep]) <= F32


@pytest.mark.parametrize("scale", [1e-12, 1e-24, 1e-30])
def test_tiny_states(scale):
    """v, states and dy whose products come near fp32's smallest numbers (1e-36 and
    more, where they hold their 24 bits)."""
    d, o, dy, dfin = make(1, 100, 4, 2, 24, 32, "f32", True, seed=96)
    d["v"] *= scale
    o["initial_states"] *= scale
    dy *= 1e-4
    dfin *= 1e-4
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, 32 ** -0.5)
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for n, w in want.items():
        assert rel(got[n].double() / scale, w / scale) <= 2 * F32, n
