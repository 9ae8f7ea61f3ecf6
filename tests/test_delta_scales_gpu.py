"""Tokens whose q and k differ by many orders of magnitude within a chunk: each
token's outputs are held to the path's accuracy by themselves.  y_t is linear in
q_t, so a small q_t has a small y_t whose relative error is the same; keys are
small only where what they write and read is small too."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import delta, delta_grads
from test_delta_gpu import make, ref_args, tol

pytestmark = pytest.mark.gpu

CASES = [(1, 100, 4, 2, 32, 64), (1, 70, 2, 1, 64, 128), (2, 65, 2, 2, 24, 200)]
ids = "b{0[0]}_L{0[1]}_H{0[2]}_G{0[3]}_P{0[4]}_N{0[5]}".format


def spread(case, dtype, most, names):
    """Inputs whose rows of `names` are brought to between 1 and 2^-most, by powers of two."""
    d, o, dy, dfin = make(*case, dtype, True, seed=50)
    gen = torch.Generator().manual_seed(51)
    for n in names:
        e = torch.randint(0, most + 1, (*d[n].shape[:3], 1), generator=gen).cuda()
        e[:, 0::9] = 0                     # the largest in every chunk
        d[n] *= torch.exp2(-e.float()).to(d[n].dtype)
    return d, o, dy, dfin


def by_token(x, ref):
    """Largest over tokens of the 2-norm of the difference over that of the reference."""
    x, ref = x.double(), ref.to(x.device)
    return ((x - ref).flatten(2).norm(dim=-1) / ref.flatten(2).norm(dim=-1)).max().item()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_small_queries(case, dtype):
    """Queries down to 2^-20 of the largest beside them."""
    d, o, dy, dfin = spread(case, dtype, 20, ("q",))
    y, _ = ssd.delta_fwd(**d, **o)
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, case[-1] ** -0.5)
    assert by_token(y, delta(*a, **kw)[0]) <= tol(y)
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for n in ("dq", "dv"):
        assert by_token(got[n], want[n]) <= 4 * tol(got[n]), n   # sums of a few hundred terms of either sign


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_small_keys(case):
    """Keys of 2^-20 beside keys of 1, in columns of their own, which alone the
    queries read.  What is left is the state's operand: a row of it is held to
    2^-25 where the bound of its magnitudes lies below 2^15.  The bound is at
    most 64 (tokens times k below 2) x 2 (a power of two above R) x 2 x 2.5 (one
    above the row sums of the inverse, 1 + 16 x 0.1 here) = 2^9.3 a chunk above
    the largest value, 2^11 after four: 2^-29 of the row's largest value.  The
    small columns' values are 2^-20 of it times some 2^-3 (a seventh of the
    tokens, and the root mean square of their sum against the largest), so 2^-6
    of them.  (With k scaled by a chunk's largest, an error of half of y.)"""
    b, L, H, G, P, N = case
    d, o, _, _ = make(*case, "f32", False, seed=52)
    half = N // 2
    small = torch.zeros(L, dtype=torch.bool)
    small[3::7] = True
    d["k"][:, small, :, :half] = 0
    d["k"][:, ~small, :, half:] = 0
    d["k"][:, small] *= 2.0 ** -20
    d["q"][:, :, :, :half] = 0               # answers with what the small keys have written
    y, _ = ssd.delta_fwd(**d, **o)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, N ** -0.5)
    ref = delta(*a, **kw)[0]
    assert not y[:, :3].any() and not ref[:, :3].any()
    assert by_token(y[:, 3:], ref[:, 3:]) <= 2.0 ** -6
