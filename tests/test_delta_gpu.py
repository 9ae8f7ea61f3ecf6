"""The gated delta rule (forward, decode step, backward) against the 64-bit
token recurrence.

Tolerances (relative 2-norm).  The products' operands carry 22 bits and the
sums 24; a result passes some 10 such roundings on its way (the products with
S, (I + A)^-1, the state's update), carried on by a recurrence that does not
amplify them here: 1e-5 is 40 times 2^-22, the framework's bound for its fp32
paths.  A bf16 result is rounded once (at most 2^-8) from a sum whose terms
were rounded to 11 bits (at most 2 x 2^-11, with independent signs): 2^-8 +
2^-10."""
import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from delta_ref import delta, delta_grads, rel

pytestmark = pytest.mark.gpu

F32 = 1e-5
BF16 = 2.0 ** -8 + 2.0 ** -10
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tol(t):
    return BF16 if t.dtype == torch.bfloat16 else F32


def make(b, L, H, G, P, N, dtype, h0=False, seed=0, lens=None, ids=None, g_max=0.5):
    gen = torch.Generator().manual_seed(seed * 7919 + L * 31 + P * 7 + N)
    t = DT[dtype]
    unit = torch.nn.functional.normalize
    d = dict(q=unit(torch.randn(b, L, G, N, generator=gen), dim=-1).to(t),
             k=unit(torch.randn(b, L, G, N, generator=gen), dim=-1).to(t),
             v=torch.randn(b, L, H, P, generator=gen).to(t),
             g=-g_max * torch.rand(b, L, H, generator=gen), beta=torch.rand(b, L, H, generator=gen))
    d = {n: x.cuda() for n, x in d.items()}
    o = dict(initial_states=torch.randn(b, H, P, N, generator=gen).cuda() if h0 else None, seq_idx=None, num_seqs=None)
    if lens is not None:
        ids = ids if ids is not None else list(range(sum(len(r) for r in lens)))
        it = iter(ids)
        o["seq_idx"] = torch.tensor([[i for n in row for i in [next(it)] * n] for row in lens], dtype=torch.int32).cuda()
        o["num_seqs"] = max(ids) + 1
    dy = torch.randn(b, L, H, P, generator=gen).to(t).cuda()
    rows = b if lens is None else o["num_seqs"]
    dfin = torch.randn(rows, H, P, N, generator=gen).cuda()
    return d, o, dy, dfin


def ref_args(d, o, scale):
    return [d[n] for n in ("q", "k", "v", "g", "beta")], dict(scale=scale, h0=o["initial_states"], seq_idx=o["seq_idx"],
                                                              num_seqs=o["num_seqs"])


def check_fwd(d, o, scale=None):
    y, f = ssd.delta_fwd(**d, **o, scale=scale)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, d["q"].shape[-1] ** -0.5 if scale is None else scale)
    yr, fr = delta(*a, **kw)
    assert rel(y, yr) <= tol(y), rel(y, yr)
    assert rel(f, fr) <= F32, rel(f, fr)
    return y, f


def check_bwd(d, o, dy, dfin, scale=None, fac=1.0):
    s = d["q"].shape[-1] ** -0.5 if scale is None else scale
    got = ssd.delta_bwd(**d, dy=dy, **o, scale=scale, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, s)
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for n, w in want.items():
        assert rel(got[n], w) <= fac * tol(got[n]), (n, rel(got[n], w))
    return got


SHAPES = [
    # b, L, H, G, P, N, dtype, h0
    (1, 1, 1, 1, 1, 1, "f32", False),
    (2, 1, 4, 2, 64, 128, "bf16", True),
    (1, 2, 2, 1, 16, 16, "bf16", False),
    (1, 31, 2, 2, 64, 64, "f32", True),
    (1, 32, 2, 1, 64, 128, "bf16", False),
    (2, 33, 2, 1, 64, 128, "bf16", True),
    (1, 64, 3, 3, 40, 72, "f32", True),
    (1, 65, 6, 2, 128, 128, "bf16", True),
    (1, 129, 2, 1, 7, 9, "bf16", True),       # rows on odd addresses
    (2, 97, 3, 1, 5, 3, "f32", True),
    (1, 100, 2, 1, 65, 100, "bf16", False),   # one row past a slice
    (1, 70, 2, 1, 200, 256, "bf16", True),
    (1, 70, 2, 2, 136, 200, "f32", True),
    (1, 300, 8, 1, 64, 128, "bf16", False),
    (3, 200, 5, 5, 24, 130, "bf16", True),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "b{}_L{}_H{}_G{}_P{}_N{}_{}_{}".format(*c))
def test_forward(case):
    d, o, _, _ = make(*case)
    check_fwd(d, o)


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "b{}_L{}_H{}_G{}_P{}_N{}_{}_{}".format(*c))
def test_backward(case):
    d, o, dy, dfin = make(*case, seed=1)
    check_bwd(d, o, dy, dfin)
    check_bwd(d, o, dy, None)


PACKED = [
    ([[1]], None), ([[1, 1, 1]], None), ([[32, 1, 33, 64]], None), ([[5, 64, 65, 96, 31]], None),
    ([[40, 30], [70], [1, 69]], None),
    ([[20, 50, 30]], [4, 0, 2]),           # out of order, ids 1 and 3 do not occur
]


@pytest.mark.parametrize("lens,ids", PACKED)
@pytest.mark.parametrize("dtype,h0", [("bf16", False), ("f32", True)])
def test_packed(lens, ids, dtype, h0):
    b, L = len(lens), sum(lens[0])
    d, o, dy, dfin = make(b, L, 4, 2, 48, 64, dtype, h0, seed=2, lens=lens, ids=ids)
    _, f = check_fwd(d, o)
    if ids is not None:
        assert not f[1].any() and not f[3].any()
    check_bwd(d, o, dy, dfin)


def test_many_short_sequences():
    lens = [[1 + (7 * i) % 5 for i in range(700)]]
    d, o, dy, dfin = make(1, sum(lens[0]), 2, 1, 16, 16, "bf16", seed=3, lens=lens)
    check_fwd(d, o)
    check_bwd(d, o, dy, dfin)


def test_more_runs_than_ids_stay_in_bounds():
    """ids that come back break the precondition: outputs are undefined, but
    nothing outside them is written and the next call is not affected."""
    d, o, dy, dfin = make(1, 90, 2, 1, 16, 16, "bf16", seed=4, lens=[[30, 30, 30]])
    bad = o["seq_idx"].clone()
    bad[0, 60:] = 0
    n = 2 * 2 * 16 * 16
    pool = torch.full((n + 512,), 7.0, device="cuda")
    ssd.delta_fwd(**d, seq_idx=bad, num_seqs=2, final_states=pool[256:256 + n].view(2, 2, 16, 16))
    ssd.delta_bwd(**d, dy=dy, seq_idx=bad, num_seqs=2, dfinal_states=dfin[:2].contiguous())
    torch.cuda.synchronize()
    assert (pool[:256] == 7).all() and (pool[256 + n:] == 7).all()
    with pytest.raises(ssd.SSDError):
        ssd.delta_fwd(**d, seq_idx=bad, num_seqs=2, check_seq=True)
    bad[0, 30:60] = 55  # an id out of range
    ssd.delta_fwd(**d, seq_idx=bad, num_seqs=2)
    torch.cuda.synchronize()
    check_fwd(d, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_and_extremes_of_decay(dtype):
    d, o, dy, dfin = make(1, 100, 3, 1, 32, 64, dtype, True, seed=5)
    d["g"][:, ::17, 0] = -torch.inf        # a decay of zero
    d["g"][:, 40:60, 0] = -200.0           # far below what exp tells from zero
    d["g"][:, :, 1] = 0.0                  # no decay
    d["g"][:, :, 2] = -5.0                 # a chunk's decay beyond 2^100
    check_fwd(d, o)
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, 64 ** -0.5)
    dg = d["g"].clone()
    dg[dg == -torch.inf] = -1e4            # the same numbers, without inf - inf in the reference
    a[3] = dg
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for n, w in want.items():
        assert rel(got[n], w) <= tol(got[n]), (n, rel(got[n], w))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extremes_of_beta_and_magnitude(dtype):
    d, o, dy, dfin = make(1, 90, 3, 3, 32, 64, dtype, True, seed=6)
    d["beta"][:, :, 0] = 0.0               # no token is written
    d["beta"][:, ::3, 1] = 0.0
    d["beta"][:, 1::3, 1] = 1.0
    d["v"][:, :, 2] *= 1e30
    d["k"][:, 7:9] = 0.0                   # a key of zero
    d["q"][:, 11] = 0.0
    y, f = ssd.delta_fwd(**d, **o)
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, 64 ** -0.5)
    yr, fr = delta(*a, **kw)
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for h in range(3):                     # each head for itself: one is 1e30 times the others
        assert rel(y[:, :, h], yr[:, :, h]) <= tol(y)
        assert rel(f[:, h], fr[:, h]) <= F32
        for n, w in want.items():
            x, r = (t[:, h] if n == "dinitial_states" else t[:, :, h] for t in (got[n], w))
            assert rel(x, r) <= tol(x), (n, h, rel(x, r))


def test_equal_keys_with_beta_one():
    """A is all ones below the diagonal: its inverse's rows cancel to two
    entries, where sums of powers of A would reach 1e18."""
    d, o, dy, dfin = make(1, 80, 2, 1, 32, 64, "f32", True, seed=7)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1.0
    d["g"][:, :, 0] = 0.0
    check_fwd(d, o)
    # dbeta and dg of this system cancel by two orders: their terms are of the size of |d| |e|
    got = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    a, kw = ref_args(d, o, 64 ** -0.5)
    want = delta_grads(*a, dy, **kw, dfin=dfin)
    for n in ("dq", "dk", "dv", "dinitial_states"):
        assert rel(got[n], want[n]) <= F32, (n, rel(got[n], want[n]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_off_16_byte_boundaries_and_guards(dtype):
    """Tensors that start in the middle of a larger one; what lies around the outputs stays."""
    d, o, dy, dfin = make(1, 75, 2, 1, 24, 40, dtype, True, seed=8)
    off = {}
    for n, t in d.items():
        pool = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        off[n] = pool[1:].view(t.shape).copy_(t)
    y0, f0 = check_fwd(off, o)
    pool = torch.full((y0.numel() + 2,), 3.0, dtype=y0.dtype, device="cuda")
    y1, f1 = ssd.delta_fwd(**off, **o, y=pool[1:-1].view(y0.shape))
    torch.cuda.synchronize()
    assert pool[0] == 3 and pool[-1] == 3
    assert torch.equal(y0, y1) and torch.equal(f0, f1)
    check_bwd(off, o, dy, dfin)


def test_calls_repeat_to_the_bit():
    d, o, dy, dfin = make(2, 200, 8, 2, 64, 128, "bf16", True, seed=9)
    a, b = ssd.delta_fwd(**d, **o), ssd.delta_fwd(**d, **o)
    x, y = (ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert all(torch.equal(x[n], y[n]) for n in x)


def test_two_streams_at_once():
    d, o, dy, dfin = make(1, 400, 8, 2, 64, 128, "bf16", True, seed=10)
    e, p, ey, efin = make(1, 300, 8, 2, 64, 128, "bf16", True, seed=11)
    want = ssd.delta_fwd(**d, **o), ssd.delta_fwd(**e, **p), ssd.delta_bwd(**e, dy=ey, **p)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            x = ssd.delta_fwd(**d, **o)
        with torch.cuda.stream(t):
            y = ssd.delta_fwd(**e, **p)
            z = ssd.delta_bwd(**e, dy=ey, **p)
        torch.cuda.synchronize()
        assert all(torch.equal(u, w) for u, w in zip(x, want[0]))
        assert all(torch.equal(u, w) for u, w in zip(y, want[1]))
        assert all(torch.equal(z[n], want[2][n]) for n in z)


@pytest.mark.parametrize("packed", [False, True])
def test_captured_and_replayed_on_new_inputs(packed):
    lens = [[100, 1, 59]] if packed else None
    d, o, dy, dfin = make(1, 160, 4, 2, 64, 64, "bf16", True, seed=12, lens=lens)
    e, p, ey, _ = make(1, 160, 4, 2, 64, 64, "bf16", True, seed=13, lens=lens)
    ssd.delta_fwd(**d, **o)
    ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, f = ssd.delta_fwd(**d, **o)
        g = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    for n in d:
        d[n].copy_(e[n])
    dy.copy_(ey)
    graph.replay()
    torch.cuda.synchronize()
    want = ssd.delta_fwd(**d, **o)
    wg = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin)
    assert torch.equal(y, want[0]) and torch.equal(f, want[1])
    assert all(torch.equal(g[n], wg[n]) for n in wg)


# ------------------------------------------------------------------ decode
STEPS = [(1, 4, 2, 64, 128, "bf16"), (3, 6, 3, 40, 72, "f32"), (2, 4, 1, 7, 4, "bf16"), (1, 2, 2, 130, 256, "f32"),
         (2, 3, 1, 33, 20, "bf16"), (70, 8, 1, 64, 128, "bf16"), (300, 2, 2, 16, 16, "f32"), (1, 1, 1, 1, 132, "f32")]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "b{}_H{}_G{}_P{}_N{}_{}".format(*c))
def test_step(case):
    b, H, G, P, N, dtype = case
    d, o, _, _ = make(b, 1, H, G, P, N, dtype, True, seed=14)
    d["g"][0, 0, 0] = -torch.inf
    a, kw = ref_args(d, o, 0.3)
    a[3] = a[3].clamp(min=-1e4)
    yr, fr = delta(*a, **kw)
    s = {n: t[:, 0].contiguous() for n, t in d.items()}
    state = o["initial_states"].clone()
    state[0, 0] *= 2                       # a finite state under a decay of zero
    y = ssd.delta_step(**s, state=state, scale=0.3)
    torch.cuda.synchronize()
    # fp32 throughout: sums of up to 256 terms
    assert rel(state, fr) <= 1e-6 and rel(y, yr[:, 0]) <= (BF16 if dtype == "bf16" else 2e-6)


def test_step_keeps_other_rows_and_reads_misaligned_v():
    d, o, _, _ = make(2, 1, 2, 1, 18, 8, "bf16", True, seed=15)
    s = {n: t[:, 0].contiguous() for n, t in d.items()}
    pool = torch.empty(s["v"].numel() + 1, dtype=torch.bfloat16, device="cuda")
    v = pool[1:].view(s["v"].shape).copy_(s["v"])
    st = torch.full((4, 2, 18, 8), 5.0, device="cuda")
    st[1:3] = o["initial_states"]
    want = o["initial_states"].clone()
    y0 = ssd.delta_step(**s, state=want)
    y1 = ssd.delta_step(s["q"], s["k"], v, s["g"], s["beta"], st[1:3])
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(st[1:3], want) and (st[0] == 5).all() and (st[3] == 5).all()


# ------------------------------------------------------------------ autograd, and a run of them together
def test_gradients_against_differences():
    """<gradient, direction> of delta_chunked against central differences of the
    64-bit recurrence.  The quotient's own error is ~eps^2 (1e-8) plus
    2^-53 / eps; the gradient's is F32 relative to |gradient| |direction|."""
    d, o, dy, dfin = make(1, 70, 4, 2, 24, 32, "f32", True, seed=16)
    leaves = {n: t.clone().requires_grad_() for n, t in d.items()}
    h0 = o["initial_states"].clone().requires_grad_()
    y, f = ssd.delta_chunked(**leaves, initial_states=h0)
    ((y * dy).sum() + (f * dfin).sum()).backward()
    for n, leaf in list(leaves.items()) + [("h0", h0)]:
        u = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(1)).cuda().double()
        u /= u.norm()

        def loss(eps):
            x = {m: t.double() for m, t in d.items()}
            s = o["initial_states"].double()
            if n == "h0":
                s = s + eps * u
            else:
                x[n] = x[n] + eps * u
            yy, ff = delta(*(x[m] for m in ("q", "k", "v", "g", "beta")), 32 ** -0.5, s)
            return ((yy * dy.double()).sum() + (ff * dfin.double()).sum()).item()

        eps = 1e-4
        quotient = (loss(eps) - loss(-eps)) / (2 * eps)
        got = (leaf.grad.double() * u).sum().item()
        assert abs(got - quotient) <= (F32 + 1e-6) * leaf.grad.norm().item() + 1e-6, (n, got, quotient)


def test_block_prefill_equals_decode_and_trains():
    """conv1d + SiLU, the delta rule and the gated norm as a block uses them:
    token by token (decode) against the whole sequence, then its gradients
    against the plain 64-bit forms of the delta rule and the norm."""
    from delta_ref import norm
    b, L, H, G, P, N = 2, 50, 4, 2, 32, 64
    gen = torch.Generator().manual_seed(17)
    C = 2 * G * N + H * P
    u = torch.randn(b, L, C, generator=gen).cuda()
    cw, cb = torch.randn(C, 4, generator=gen).cuda() * 0.5, torch.randn(C, generator=gen).cuda() * 0.1
    w, bias = torch.rand(P, generator=gen).cuda() + 0.5, torch.randn(P, generator=gen).cuda()
    g, beta = -0.3 * torch.rand(b, L, H, generator=gen).cuda(), torch.rand(b, L, H, generator=gen).cuda()
    z = torch.randn(b, L, H, P, generator=gen).cuda()

    def split(x):
        q, k, v = x.split([G * N, G * N, H * P], -1)
        unit = torch.nn.functional.normalize
        return (unit(q.reshape(b, -1, G, N), dim=-1), unit(k.reshape(b, -1, G, N), dim=-1),
                v.reshape(b, -1, H, P).contiguous())

    xin = u.clone().requires_grad_()
    x = ssd.causal_conv1d_silu(xin, cw, cb)
    q, k, v = split(x)
    gl, bl, zl, wl = (t.clone().requires_grad_() for t in (g, beta, z, w))
    y, fin = ssd.delta_chunked(q, k, v, gl, bl)
    out = ssd.gated_layer_norm(y, wl, bias, z=zl)
    state = torch.zeros(b, H, P, N, device="cuda")
    with torch.no_grad():
        for t in range(L):
            yt = ssd.delta_step(*(a[:, t].contiguous() for a in (q, k, v, g, beta)), state)
            ot = ssd.layer_norm(yt, w, bias, z=z[:, t].contiguous())
            # both sides are off by F32 before the norm, which divides by the row's deviation
            assert rel(ot, out[:, t]) <= 1e-4
    assert rel(state, fin) <= F32
    dout = torch.randn(out.shape, generator=gen).cuda()
    out.backward(dout)

    xr = u.double().requires_grad_()
    pad = torch.nn.functional.pad(xr.transpose(1, 2), (3, 0))
    c = torch.nn.functional.conv1d(pad, cw.double().unsqueeze(1), cb.double(), groups=C).transpose(1, 2)
    qr, kr, vr = split(c * torch.sigmoid(c))
    gr, br, zr, wr = (t.double().requires_grad_() for t in (g, beta, z, w))
    yr, _ = delta(qr, kr, vr, gr, br, N ** -0.5)
    norm(yr, wr, bias, 1e-5, zr).backward(dout.double())
    for got, want in ((xin, xr), (gl, gr), (bl, br), (zl, zr), (wl, wr)):
        assert rel(got.grad, want.grad) <= 1e-4, rel(got.grad, want.grad)  # as above, through the norm


# ------------------------------------------------------------------ the far ends
def test_offsets_past_32_bits():
    """66000 tokens of 512 heads: v, y, the tiles, E, D and the checkpointed
    states pass 2^31 elements.  The last group's heads do not depend on the
    others, so a call of them alone, whose offsets are small, gives the same bits."""
    L, H, G, P, N = 66000, 512, 8, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(17)
    d = {n: torch.randn(1, L, x, m, generator=gen, device="cuda", dtype=torch.bfloat16) * s
         for n, x, m, s in (("q", G, N, 0.09), ("k", G, N, 0.09), ("v", H, P, 1.0))}
    d["g"] = -0.3 * torch.rand(1, L, H, generator=gen, device="cuda")
    d["beta"] = torch.rand(1, L, H, generator=gen, device="cuda")
    dy = torch.randn(1, L, H, P, generator=gen, device="cuda", dtype=torch.bfloat16)
    assert d["v"].numel() > 2 ** 31
    last = {n: t[:, :, -(t.shape[2] // G):].contiguous() for n, t in d.items()}
    y, f = ssd.delta_fwd(**d)
    ys, fs = ssd.delta_fwd(**last)
    hs = H // G
    assert torch.isfinite(ys).all() and torch.equal(y[:, :, -hs:], ys) and torch.equal(f[:, -hs:], fs)
    del y, ys
    got = ssd.delta_bwd(**d, dy=dy)
    want = ssd.delta_bwd(**last, dy=dy[:, :, -hs:].contiguous())
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n][:, :, -want[n].shape[2]:], want[n]), n
    torch.cuda.empty_cache()


def test_step_offsets_past_32_bits():
    b, H, P, N = 4096, 80, 64, 128
    d, o, _, _ = make(1, 1, H, 1, P, N, "bf16", True, seed=18)
    s = {n: t[:, 0].contiguous() for n, t in d.items()}
    state = torch.zeros(b, H, P, N, device="cuda")
    assert state.numel() > 2 ** 31
    state[-1] = o["initial_states"][0]
    many = {n: t.expand(b, *t.shape[1:]).contiguous() for n, t in s.items()}
    y = ssd.delta_step(**many, state=state)
    one = o["initial_states"].clone()
    assert torch.equal(ssd.delta_step(**s, state=one)[0], y[-1]) and torch.equal(state[-1], one[0])
    del state
    torch.cuda.empty_cache()


def test_many_ids():
    """More ids than are ranked (2048) and more tokens than the run list keeps
    flags of (65536), rows of different packing; most ids do not occur."""
    lens = [[1 + (5 * i) % 31 for i in range(2600)], []]
    L = sum(lens[0])
    lens[1] = [7, L - 7]
    ids = [3 * i for i in range(2602)]
    assert 2 * L > 65536
    d, o, dy, dfin = make(2, L, 2, 1, 16, 16, "bf16", True, seed=19, lens=lens, ids=ids)
    o["num_seqs"] += 100
    dfin = torch.cat([dfin, dfin[:100]])
    _, f = check_fwd(d, o)
    assert not f[1].any() and not f[-1].any()
    check_bwd(d, o, dy, dfin)


def test_initial_gradient_without_initial_states():
    d, o, dy, dfin = make(2, 90, 4, 2, 16, 32, "f32", True, seed=20)
    z = dict(o, initial_states=torch.zeros_like(o["initial_states"]))
    got = ssd.delta_bwd(**d, dy=dy, dfinal_states=dfin, want_dinitial_states=True)
    want = ssd.delta_bwd(**d, dy=dy, **z, dfinal_states=dfin)
    assert torch.equal(got["dinitial_states"], want["dinitial_states"])
    assert all(rel(got[n], want[n]) <= F32 for n in got)


def test_two_host_threads():
    from concurrent.futures import ThreadPoolExecutor
    sets = [make(1, 200 + 50 * i, 4, 2, 64, 64, "bf16", True, seed=21 + i) for i in range(2)]
    want = [ssd.delta_fwd(**d, **o) for d, o, _, _ in sets]
    torch.cuda.synchronize()

    def run(i):
        d, o, _, _ = sets[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            r = [ssd.delta_fwd(**d, **o) for _ in range(20)]
            torch.cuda.current_stream().synchronize()
        return all(torch.equal(x, w) for p in r for x, w in zip(p, want[i]))

    with ThreadPoolExecutor(2) as pool:
        assert all(pool.map(run, range(2)))


def test_training_step_captured():
    """Forward and backward of both operators in one graph, replayed on new inputs."""
    def step(v, w, rest):
        y, _ = ssd.delta_chunked(rest["q"], rest["k"], v, rest["g"], rest["beta"])
        return torch.autograd.grad((ssd.gated_layer_norm(y, w).float() ** 3).sum(), (v, w))

    d, _, _, _ = make(1, 100, 4, 2, 64, 64, "bf16", seed=23)
    e, _, _, _ = make(1, 100, 4, 2, 64, 64, "bf16", seed=24)
    v, w = d["v"].requires_grad_(), torch.rand(64, device="cuda").requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(v, w, d)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(v, w, d)
    with torch.no_grad():
        for n in d:
            d[n].copy_(e[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, step(v, w, d)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_batch(dtype):
    """Rows of 100, 33 and 1 tokens padded to 130: padding with g and beta zero
    neither reaches back nor moves the state, whatever q, k and v hold there."""
    d, o, dy, dfin = make(3, 130, 4, 2, 24, 32, dtype, True, seed=25)
    lens = [100, 33, 1]
    for i, n in enumerate(lens):
        d["g"][i, n:] = 0
        d["beta"][i, n:] = 0
        dy[i, n:] = 0
    y, f = ssd.delta_fwd(**d, initial_states=o["initial_states"])
    got = ssd.delta_bwd(**d, dy=dy, initial_states=o["initial_states"], dfinal_states=dfin)
    for i, n in enumerate(lens):
        one = {m: t[i:i + 1, :n].contiguous() for m, t in d.items()}
        h0 = o["initial_states"][i:i + 1].contiguous()
        ys, fs = ssd.delta_fwd(**one, initial_states=h0)
        # both are within the tolerance of the same recurrence
        assert rel(y[i:i + 1, :n], ys) <= 2 * tol(ys) and rel(f[i:i + 1], fs) <= 2 * F32
        want = ssd.delta_bwd(**one, dy=dy[i:i + 1, :n].contiguous(), initial_states=h0, dfinal_states=dfin[i:i + 1].contiguous())
        for m in ("dq", "dk", "dv", "dg", "dbeta"):
            assert rel(got[m][i:i + 1, :n], want[m]) <= 2 * tol(want[m]), m
        assert rel(got["dinitial_states"][i:i + 1], want["dinitial_states"]) <= 2 * F32
