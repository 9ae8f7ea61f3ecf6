"""Rows whose mean is far larger than what they deviate from it: the mean's own
rounding must not show in the outputs."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import norm, rel

pytestmark = pytest.mark.gpu

COLS = [3, 7, 40, 64, 129, 300, 1000, 1025, 2047, 2560, 4100, 5120, 8200, 10240, 20001]
DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_values_are_the_bias(cols, dtype):
    """x - mean is exact next to the mean, and so the same for all columns of a
    row; its mean, taken out again, leaves what rounding left of it: (some 100 x
    2^-24)^2 of x at the most (the longest chain of a sum has 80 terms), times
    eps^-1/2."""
    value = torch.tensor([1000.0, -30000.0, 1234.567, 0.1, -7.25, 1e5], device="cuda").to(dtype)
    x = value[:, None].expand(6, cols).contiguous()
    gen = torch.Generator().manual_seed(cols)
    w, b = torch.randn(cols, generator=gen).cuda(), torch.randn(cols, generator=gen).cuda()
    y = ssd.layer_norm(x, w, b)
    dy = torch.randn(6, cols, generator=gen).to(dtype).cuda()
    dx, dw, db, _ = ssd.layer_norm_bwd(x, w, b, dy)
    torch.cuda.synchronize()
    n = (100 * 2.0 ** -24) ** 2 * value.double().abs()[:, None] * 1e-5 ** -0.5
    step = torch.finfo(dtype).eps / 2
    assert ((y.double() - b.double()).abs() <= n * w.double().abs() + step * b.double().abs()).all(), \
        (y.double() - b.double()).abs().max().item()
    assert (dw.double().abs() <= 2 * (n * dy.double().abs()).sum(0) + 1e-30).all()
    lim = 2.0 ** -8 if dtype == torch.bfloat16 else 2e-6
    assert rel(db, dy.double().sum(0)) <= 1e-5
    h = dy.double() * w.double()
    # dx = rstd (hw - mean(hw)) with n = 0: rstd is exactly eps^-1/2 but for rounding
    assert rel(dx, (h - h.mean(-1, keepdim=True)) * 1e-5 ** -0.5) <= 2 * lim


@pytest.mark.parametrize("cols", COLS[1:])
def test_small_deviations_from_a_large_mean(cols):
    """fp32 rows of mean 1e4 and deviation 1, against the norm of those same
    values: x - mean is exact, so only the sums' rounding is left (2e-6, as for
    rows without a mean; twice it for the gradients, through n)."""
    gen = torch.Generator().manual_seed(cols)
    x = (torch.randn(40, cols, generator=gen) + 1e4).cuda()
    w, b = torch.randn(cols, generator=gen).cuda(), torch.randn(cols, generator=gen).cuda()
    dy = torch.randn(40, cols, generator=gen).cuda()
    y = ssd.layer_norm(x, w, b)
    dx, dw, _, _ = ssd.layer_norm_bwd(x, w, b, dy)
    torch.cuda.synchronize()
    xr, wr = x.double().requires_grad_(), w.double().requires_grad_()
    ref = norm(xr, wr, b)
    gx, gw = torch.autograd.grad(ref, (xr, wr), dy.double())
    assert rel(y, ref) <= 2e-6 and rel(dx, gx) <= 4e-6 and rel(dw, gw) <= 1e-5
