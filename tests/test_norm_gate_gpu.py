"""SiLU of the gated norm element by element, over every z that a gate can hold:
a far one must not lose its own relative accuracy, which the 2-norm of a tensor
does not see."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd

pytestmark = pytest.mark.gpu

# a few units: the exponential (2 of 2^-23), 1 + t and the divide (2), the products with z and with the norm (1 each);
# in bf16 the exponential's argument is rounded as well (2^-24 of at most 100), which its result's rounding hides
FEW = {torch.float32: 8 * 2.0 ** -23, torch.bfloat16: 8 * 2.0 ** -23 + 100 * 1.45 * 2.0 ** -24}


def gated(dtype, cols):
    """x with a norm of +-1 exactly (up to eps), z from -100 to 30."""
    n = 131 * cols
    z = torch.linspace(-100.0, 30.0, n, dtype=torch.float64).to(dtype).view(131, cols).cuda()
    x = torch.ones(131, cols, dtype=dtype, device="cuda")
    x[:, ::2] = -1
    return x, z


@pytest.mark.parametrize("cols", [64, 130, 1030, 2048, 4100, 5120, 10240])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_silu(dtype, cols):
    x, z = gated(dtype, cols)
    y = ssd.layer_norm(x, eps=0.0, z=z)
    dx, _, _, dz = ssd.layer_norm_bwd(x, None, None, torch.ones_like(x), eps=0.0, z=z)
    torch.cuda.synchronize()
    zd = z.double()
    s = 1 / (1 + torch.exp(-zd))
    want = x.double() * zd * s
    few = FEW[dtype]
    step = few + (2.0 ** -8 if dtype == torch.bfloat16 else 0)
    # fp32: normal numbers.  bf16: down to z = -87; below, zero will do for what is less than 2e-36
    ok = want.abs() > 1e-37 if dtype == torch.float32 else zd > -87
    assert ok[zd < -85].any() and (y[~ok].abs() <= 2e-36).all() and (dz[~ok].abs() <= 2e-36).all()
    assert ((y.double() - want).abs()[ok] <= step * want.abs()[ok]).all(), \
        ((y.double() - want).abs() / want.abs())[ok].max().item()
    # SiLU' = s (1 + z (1 - s)): its two terms may cancel, each is off by `few`; again where it is a normal number
    slope = x.double() * s * (1 + zd * (1 - s))
    lim = step * slope.abs() + few * (s + (zd * s * (1 - s)).abs())
    ok = ok & (slope.abs() > 1e-37)
    assert ok[zd < -85].any()
    assert ((dz.double() - slope).abs()[ok] <= lim[ok]).all()
    assert torch.isfinite(dx).all()
