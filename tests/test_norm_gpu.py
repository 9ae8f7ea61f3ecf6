"""The gated layer norm and its backward against the 64-bit formula.

Tolerances (relative 2-norm): fp32 arithmetic on sums of up to 20000 terms, the
mean taken first: 2e-6 (16 x 2^-23); a bf16 result is rounded once more, by at
most 2^-8.  Column sums are fp32 partial sums of at most a few thousand terms
with random signs, added in 64 bits: 1e-5."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import norm, rel

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tol(t):
    return 2.0 ** -8 if t.dtype == torch.bfloat16 else 2e-6


def make(rows, cols, dtype, affine, gate, seed=0):
    gen = torch.Generator().manual_seed(seed * 1009 + rows * 13 + cols)
    t = DT[dtype]
    x = (torch.randn(rows, cols, generator=gen) * 1.5 + 0.3).to(t).cuda()
    w = (1 + 0.2 * torch.randn(cols, generator=gen)).cuda() if affine else None
    b = (0.1 * torch.randn(cols, generator=gen)).cuda() if affine else None
    z = torch.randn(rows, cols, generator=gen).to(t).cuda() if gate else None
    dy = torch.randn(rows, cols, generator=gen).to(t).cuda()
    return x, w, b, z, dy


def check(x, w, b, z, dy, eps=1e-5, fac=1.0):
    y = ssd.layer_norm(x, w, b, eps=eps, z=z)
    got = dict(zip(("dx", "dw", "db", "dz"), ssd.layer_norm_bwd(x, w, b, dy, eps=eps, z=z)))
    torch.cuda.synchronize()
    leaves = {n: t.double().requires_grad_() for n, t in (("dx", x), ("dw", w), ("db", b), ("dz", z)) if t is not None}
    ref = norm(leaves["dx"], leaves.get("dw"), leaves.get("db"), eps, leaves.get("dz"))
    assert rel(y, ref) <= fac * tol(y), rel(y, ref)
    for n, r in zip(leaves, torch.autograd.grad(ref, list(leaves.values()), dy.double())):
        lim = 1e-5 if n in ("dw", "db") else fac * tol(x)
        assert rel(got[n], r) <= lim, (n, rel(got[n], r))


COLS = [3, 4, 8, 31, 32, 33, 64, 96, 128, 129, 256, 300, 512, 1000, 1024, 1025, 2048, 2560, 4095, 4096, 5120, 8192,
        10240, 16384, 20001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widths(cols, dtype):
    rows = 37 if cols > 300 else 500
    check(*make(rows, cols, dtype, True, cols % 2 == 0))
    check(*make(1, cols, dtype, cols % 3 == 0, cols % 2 == 1, seed=1))


@pytest.mark.parametrize("cols", [8, 64, 129, 5120])
def test_many_rows(cols):
    check(*make(400000 // cols + 3000, cols, "bf16", True, True, seed=2))


def test_one_column_is_the_bias():
    x, w, b, z, dy = make(9, 1, "f32", True, False)
    y = ssd.layer_norm(x, w, b)
    dx, dw, db, _ = ssd.layer_norm_bwd(x, w, b, dy)
    assert torch.equal(y, b.expand(9, 1)) and not dx.any() and not dw.any() and rel(db, dy.double().sum(0)) <= 1e-6


def test_large_mean_and_constant_rows():
    """The mean is taken out before squares are summed: a mean of 1e4
    deviations costs what fp32 holds of x - mean (2^-24 x 1e4 per element)."""
    x, w, b, _, dy = make(50, 512, "f32", True, False, seed=3)
    x = x + 1e4
    y = ssd.layer_norm(x, w, b)
    assert rel(y, norm(x, w, b)) <= 1e4 * 2.0 ** -24 * 4
    x[:] = 2.5  # no deviation at all: bias
    assert torch.equal(ssd.layer_norm(x, w, b), b.expand_as(x))


def test_gate_far_out():
    x, w, b, z, dy = make(20, 64, "f32", True, True, seed=4)
    z[0], z[1], z[2] = 100.0, -100.0, -torch.inf
    y = ssd.layer_norm(x, w, b, z=z)
    ref = norm(x, w, b, 1e-5, z)
    assert torch.isfinite(y).all() and rel(y, ref) <= 2e-6 and not y[2].any()


def test_gate_far_out_backward():
    """A gate of -inf passes nothing: dz and the row's share of the rest are
    zero; and no group without a row adds to the sums (eps = 0)."""
    x, w, b, z, dy = make(3, 64, "f32", True, True, seed=9)
    z[1] = -torch.inf
    dx, dw, db, dz = ssd.layer_norm_bwd(x, w, b, dy, eps=0.0, z=z)
    assert not dx[1].any() and not dz[1].any()
    keep = [0, 2]
    want = ssd.layer_norm_bwd(x[keep], w, b, dy[keep], eps=0.0, z=z[keep])
    assert rel(dw, want[1]) <= 1e-6 and rel(db, want[2]) <= 1e-6
    for cols in (1030, 4100):  # a CTA a row, and rows swept from memory
        x, w, b, z, dy = make(3, cols, "bf16", True, True, seed=10)
        z[1] = -torch.inf
        assert not ssd.layer_norm(x, w, b, z=z)[1].any()
        got = ssd.layer_norm_bwd(x, w, b, dy, z=z)
        assert not got[0][1].any() and not got[3][1].any() and all(torch.isfinite(t).all() for t in got)


def test_shapes_strides_and_places():
    x, w, b, z, dy = make(60, 64, "bf16", True, True, seed=5)
    y = ssd.layer_norm(x, w, b, z=z)
    x5, z5 = x.view(3, 4, 5, 64), z.view(3, 4, 5, 64)
    assert torch.equal(ssd.layer_norm(x5, w, b, z=z5).view(60, 64), y)
    inplace = x.clone()
    assert torch.equal(ssd.layer_norm(inplace, w, b, z=z, out=inplace), y)
    pool = torch.full((60 * 64 + 2,), 3.0, dtype=torch.bfloat16, device="cuda")
    off = pool[1:-1].view(60, 64)
    assert torch.equal(ssd.layer_norm(x, w, b, z=z, out=off), y) and pool[0] == 3 and pool[-1] == 3
    off.copy_(x)
    g = ssd.layer_norm_bwd(off, w, b, dy, z=z)
    for p, q in zip(g, ssd.layer_norm_bwd(x, w, b, dy, z=z)):
        assert rel(p, q) <= 2.0 ** -7  # summed in another order, rounded on either side


def test_repeats_streams_and_graphs():
    x, w, b, z, dy = make(3000, 640, "bf16", True, True, seed=6)
    y, g = ssd.layer_norm(x, w, b, z=z), ssd.layer_norm_bwd(x, w, b, dy, z=z)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, g2 = ssd.layer_norm(x, w, b, z=z), ssd.layer_norm_bwd(x, w, b, dy, z=z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, g3 = ssd.layer_norm(x, w, b, z=z), ssd.layer_norm_bwd(x, w, b, dy, z=z)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)
    assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(g, g2, g3))


def test_wanted_gradients_only():
    x, w, b, z, dy = make(40, 96, "f32", True, True, seed=7)
    dx, dw, db, dz = ssd.layer_norm_bwd(x, w, b, dy, z=z, want_dweight=False, want_dbias=False)
    full = ssd.layer_norm_bwd(x, w, b, dy, z=z)
    assert dw is None and db is None and torch.equal(dx, full[0]) and torch.equal(dz, full[3])
    _, dw, db, dz = ssd.layer_norm_bwd(x, None, None, dy, want_dweight=True, want_dbias=True)
    assert dz is None and rel(db, dy.double().sum(0)) <= 1e-5


def test_gradients_against_differences():
    x, w, b, z, dy = make(11, 40, "f32", True, True, seed=8)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, z)]
    (ssd.gated_layer_norm(leaves[0], leaves[1], leaves[2], 1e-5, leaves[3]) * dy).sum().backward()
    for i, leaf in enumerate(leaves):
        u = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(i)).cuda().double()
        u /= u.norm()

        def loss(e):
            t = [a.double() + (e * u if j == i else 0) for j, a in enumerate((x, w, b, z))]
            return (norm(t[0], t[1], t[2], 1e-5, t[3]) * dy.double()).sum().item()

        q = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert abs((leaf.grad.double() * u).sum().item() - q) <= 1e-5 * leaf.grad.norm().item() + 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [7, 64, 130, 300, 1000, 1024, 2048, 5120, 8192, 16384, 20001])
def test_in_place(cols, dtype):
    """out may be x or z itself, whichever kernel the width takes."""
    x, w, b, z, _ = make(700, cols, dtype, True, True, seed=9)
    y = ssd.layer_norm(x, w, b, z=z)
    for at in (x.clone(), z.clone()):
        args = (at, z) if torch.equal(at, x) else (x, at)
        assert torch.equal(ssd.layer_norm(args[0], w, b, z=args[1], out=at), y)


@pytest.mark.parametrize("rows,cols", [(450000, 5120), (36000000, 64)])
def test_offsets_past_32_bits(rows, cols):
    x = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    w = torch.rand(cols, device="cuda")
    end = x[-100:].clone()
    assert torch.equal(ssd.layer_norm(x, w)[-100:], ssd.layer_norm(end, w))
    assert torch.equal(ssd.layer_norm_bwd(x, w, None, x)[0][-100:], ssd.layer_norm_bwd(end, w, None, end)[0])
    torch.cuda.empty_cache()
