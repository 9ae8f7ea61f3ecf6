"""The norm's backward in a workspace of exactly the size it asks for, whatever
that holds before the call; the bytes around it stay."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_03_b200 as ssd
from test_norm_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 4), (1, 5120), (3, 64), (5000, 7), (5000, 64), (30000, 8), (900, 300), (700, 1030),
                                       (600, 2048), (1000, 4096), (700, 4100), (700, 5120), (500, 8192), (3, 10240),
                                       (600, 10241)])
def test_exact_size(rows, cols, dtype, off):
    x, w, b, z, dy = make(rows, cols, dtype, True, True, seed=70)
    if off:                                    # rows that start `off` elements behind a 16-byte boundary
        pool = torch.empty(x.numel() + off, dtype=x.dtype, device="cuda")
        x = pool[off:].view(x.shape).copy_(x)
    want = ssd.layer_norm_bwd(x, w, b, dy, z=z)
    out = [torch.empty_like(t) for t in want]
    a = ssd.NormBwdArgs(rows, cols, ssd._dtype(x), 1e-5, x.data_ptr(), w.data_ptr(), b.data_ptr(), z.data_ptr(), dy.data_ptr(),
                        *(t.data_ptr() for t in out))
    n = int(ssd.lib.ssd_layer_norm_bwd_workspace_size(ctypes.byref(a)))
    for fill in (0, 255):
        pool = torch.full((n + 8192,), fill, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = pool.data_ptr() + 4096, n
        for t in out:
            t.fill_(float("nan"))
        ssd._call(ssd.lib.ssd_layer_norm_bwd, a, x.device)
        torch.cuda.synchronize()
        assert (pool[:4096] == fill).all() and (pool[4096 + n:] == fill).all()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
