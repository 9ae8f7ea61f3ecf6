"""What the delta rule returns in bf16 is the rounding of a value held to 32
bits: beyond the half step (up to 2^-8 of the value) that the one rounding may
be off by, an output is no further from the 64-bit recurrence than the fp32
path is (1e-5 in the 2-norm, as in test_delta_gpu.py)."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import delta, delta_grads
from test_delta_gpu import F32, make, ref_args

pytestmark = pytest.mark.gpu

CASES = [(1, 77, 4, 2, 64, 128, True), (2, 200, 4, 1, 64, 64, False), (1, 129, 6, 3, 128, 128, True),
         (1, 90, 2, 1, 40, 200, True), (1, 5, 2, 2, 7, 9, False)]
ids = "b{0[0]}_L{0[1]}_H{0[2]}_G{0[3]}_P{0[4]}_N{0[5]}".format


def beyond_half_a_step(x, ref):
    """2-norm of how far x is from the reference beyond half a bf16 step, relative to the reference's."""
    assert x.dtype == torch.bfloat16
    ref = ref.to(x.device)
    half = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=1e-300))) - 8)
    return ((x.double() - ref).abs() - half).clamp(min=0).norm().item() / ref.norm().item()


def test_the_measure():
    """A value rounded once has nothing beyond half a step (torch passes fp32 on
    the way from 64 bits, another 2^-24 at most); one whose terms had 11 bits has."""
    gen = torch.Generator().manual_seed(0)
    ref = torch.randn(100000, generator=gen, dtype=torch.float64)
    assert beyond_half_a_step(ref.bfloat16(), ref) <= 2.0 ** -24
    off = ref * (1 + 2.0 ** -12 * torch.randn(100000, generator=gen, dtype=torch.float64))
    assert beyond_half_a_step(off.bfloat16(), ref) > 3 * F32


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_y(case):
    b, L, H, G, P, N, h0 = case
    d, o, _, _ = make(b, L, H, G, P, N, "bf16", h0, seed=40)
    y, _ = ssd.delta_fwd(**d, **o)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, N ** -0.5)
    got = beyond_half_a_step(y, delta(*a, **kw)[0])
    assert got <= F32, got


def test_y_packed():
    d, o, _, _ = make(1, 160, 4, 2, 64, 128, "bf16", True, seed=41, lens=[[20, 33, 1, 106]])
    y, _ = ssd.delta_fwd(**d, **o)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, 128 ** -0.5)
    got = beyond_half_a_step(y, delta(*a, **kw)[0])
    assert got <= F32, got


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_gradients(case):
    b, L, H, G, P, N, h0 = case
    d, o, dy, dfin = make(b, L, H, G, P, N, "bf16", h0, seed=42)
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, N ** -0.5)
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for n in ("dq", "dk", "dv"):
        off = beyond_half_a_step(got[n], want[n])
        assert off <= F32, (n, off)
