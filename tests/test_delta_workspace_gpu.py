"""The delta rule's results do not depend on what its workspace holds before
the call: zeros, or bytes that are NaN in every type the kernels keep there.
Pieces of one chunk (1 to 32 tokens behind a multiple of 64), packed tails and
ids that do not occur are among the cases; the workspace has the size that is
asked for and lies inside a larger one whose rest must stay."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from test_delta_gpu import PACKED, SHAPES, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu

TAILS = [(1, L, 4, 2, 16, 16, "f32", False) for L in (1, 20, 32, 33, 65, 96, 97, 129)] + [
    (1, 20, 32, 8, 16, 16, "f32", True), (1, 32, 256, 256, 4, 4, "bf16", False), (2, 70, 64, 1, 16, 16, "bf16", True)]


def need(a, size):
    return int(getattr(ssd.lib, size)(ctypes.byref(a)))


def both(d, o, dy, dfin):
    a = ssd._delta_args(*(d[n] for n in ("q", "k", "v", "g", "beta")), None, o["initial_states"], o["seq_idx"], o["num_seqs"])
    fwd = need(a, "ssd_delta_fwd_workspace_size")
    b = ssd.DeltaBwdArgs(a, dy.data_ptr(), ssd._ptr(dfin))
    bwd = need(b, "ssd_delta_bwd_workspace_size")
    got = []
    for fill in (0, 255):
        pool = torch.full((max(fwd, bwd) + 2 * 4096,), fill, dtype=torch.uint8, device="cuda")
        rest = pool[:4096], pool[4096 + fwd:].clone()
        y, f = ssd.delta_fwd(**d, **o, workspace=pool[4096:4096 + fwd])
        assert torch.equal(pool[4096 + fwd:], rest[1]) and (rest[0] == fill).all()
        pool.fill_(fill)
        g = ssd.delta_bwd(**d, dy=dy, **o, dfinal_states=dfin, workspace=pool[4096:4096 + bwd])
        assert (pool[4096 + bwd:] == fill).all() and (pool[:4096] == fill).all()
        got.append({"y": y, "f": f, **{n: t for n, t in g.items() if t is not None}})
    for n in got[0]:
        assert torch.equal(got[0][n], got[1][n]), n
    for n, t in got[0].items():
        assert torch.isfinite(t).all(), n


@pytest.mark.parametrize("case", SHAPES + TAILS, ids=lambda c: "b{}_L{}_H{}_G{}_P{}_N{}_{}_{}".format(*c))
def test_any_contents(case):
    d, o, dy, dfin = make(*case, seed=30)
    both(d, o, dy, dfin)
    both(d, o, dy, None)


@pytest.mark.parametrize("lens,ids", PACKED)
@pytest.mark.parametrize("dtype,h0", [("bf16", False), ("f32", True)])
def test_any_contents_packed(lens, ids, dtype, h0):
    d, o, dy, dfin = make(len(lens), sum(lens[0]), 4, 2, 48, 64, dtype, h0, seed=31, lens=lens, ids=ids)
    both(d, o, dy, dfin)


@pytest.mark.parametrize("case", TAILS, ids=lambda c: "b{}_L{}_H{}_G{}_P{}_N{}_{}_{}".format(*c))
def test_short_tails(case):
    d, o, dy, dfin = make(*case, seed=32)
    check_fwd(d, o)
    check_bwd(d, o, dy, dfin)
