"""Rows that a norm's sums could go wrong on: with infinities and NaN, and with a
first pack far from the rest of the row."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import norm, rel
from test_norm_gpu import make

pytestmark = pytest.mark.gpu

COLS = [7, 8, 64, 130, 300, 512, 1000, 2048, 4100, 5120, 8192, 10240]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_that_is_not_finite_is_nan(cols, dtype, gate):
    """As the formula has it: an infinite mean leaves no difference, an infinite
    difference no deviation.  Rows beside it are not touched."""
    x, w, b, z, dy = make(600, cols, dtype, True, gate, seed=90)
    want = ssd.layer_norm(x, w, b, z=z), ssd.layer_norm_bwd(x, w, b, dy, z=z)
    bad = {3: (0, float("inf")), 100: (cols - 1, -float("inf")), 301: (cols // 2, float("nan")), 599: (cols // 3, float("inf"))}
    for r, (c, v) in bad.items():
        x[r, c] = v
    x[599, 0] = -float("inf")
    y = ssd.layer_norm(x, w, b, z=z)
    dx, dw, _, dz = ssd.layer_norm_bwd(x, w, b, dy, z=z)
    torch.cuda.synchronize()
    rows = torch.tensor(sorted(bad), device="cuda")
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.isnan(y[rows]).all() and torch.isnan(dx[rows]).all() and torch.isnan(dw).all()
    assert torch.equal(y[keep], want[0][keep]) and torch.equal(dx[keep], want[1][0][keep])
    if gate:
        assert torch.isnan(dz[rows]).all() and torch.equal(dz[keep], want[1][3][keep])


@pytest.mark.parametrize("cols", [520, 1024, 2048, 5120, 8192])
def test_first_pack_far_from_the_rest(cols):
    """The sums are of differences to the mean of the row's first eight values:
    with those far out, var = mean((x - K)^2) - mean(x - K)^2 cancels by cols / 8
    at the most.  Of 24 bits that leaves 2^-24 cols / 8 <= 2^-14 of var, half of it
    in rstd, beside one rounding to bf16."""
    gen = torch.Generator().manual_seed(cols)
    x = torch.randn(30, cols, generator=gen)
    x[:10, :8] += 1000.0
    x[10:20, :8] = 50.0
    x[20:, :8] = torch.tensor([1e6, -1e6] * 4)
    x, w, b = x.bfloat16().cuda(), torch.randn(cols, generator=gen).cuda(), torch.randn(cols, generator=gen).cuda()
    dy = torch.randn(30, cols, generator=gen).bfloat16().cuda()
    y, g = ssd.layer_norm(x, w, b), ssd.layer_norm_bwd(x, w, b, dy)
    torch.cuda.synchronize()
    xr = x.double().requires_grad_()
    ref = norm(xr, w, b)
    dx = torch.autograd.grad(ref, xr, dy.double())[0]
    for r in range(3):
        s = slice(10 * r, 10 * r + 10)
        assert rel(y[s], ref[s]) <= 2.0 ** -8 + 2.0 ** -14 and rel(g[0][s], dx[s]) <= 2.0 ** -8 + 2.0 ** -13
