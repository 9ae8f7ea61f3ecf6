"""Plain 64-bit references of the gated delta rule and the gated layer norm,
token by token, for the tests (torch, any device)."""
import torch


def runs_of(seq_idx, b, L):
    """(row, first token, length, id) of every maximal run, in order."""
    out = []
    for r in range(b):
        t = 0
        while t < L:
            e = t + 1
            if seq_idx is not None:
                while e < L and seq_idx[r, e] == seq_idx[r, t]:
                    e += 1
            else:
                e = L
            out.append((r, t, e - t, r if seq_idx is None else int(seq_idx[r, t])))
            t = e
    return out


def delta(q, k, v, g, beta, scale, h0=None, seq_idx=None, num_seqs=None):
    """(y, final_states) in 64 bits; differentiable."""
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    b, L, H, P = v.shape
    G, N = q.shape[2:]
    q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
    seq = None if seq_idx is None else seq_idx.cpu()
    ys = [[None] * L for _ in range(b)]
    rows = b if seq_idx is None else num_seqs
    fin = [torch.zeros(H, P, N, dtype=torch.float64, device=v.device)] * rows
    for r, t0, n, i in runs_of(seq, b, L):
        S = torch.zeros(H, P, N, dtype=torch.float64, device=v.device)
        if h0 is not None and t0 == 0:
            S = h0[r].double()
        for t in range(t0, t0 + n):
            S = S * g[r, t].exp()[:, None, None]
            u = beta[r, t][:, None] * (v[r, t] - (S @ k[r, t].unsqueeze(-1)).squeeze(-1))
            S = S + u.unsqueeze(-1) * k[r, t].unsqueeze(1)
            ys[r][t] = scale * (S @ q[r, t].unsqueeze(-1)).squeeze(-1)
        fin[i] = S
    return torch.stack([torch.stack(y) for y in ys]), torch.stack(fin)


def delta_grads(q, k, v, g, beta, dy, scale, h0=None, seq_idx=None, num_seqs=None, dfin=None):
    leaves = [t.detach().double().requires_grad_() for t in (q, k, v, g, beta)]
    if h0 is not None:
        leaves.append(h0.detach().double().requires_grad_())
    y, fin = delta(*leaves[:5], scale, leaves[5] if h0 is not None else None, seq_idx, num_seqs)
    loss = (y * dy.double()).sum() + (0 if dfin is None else (fin * dfin.double()).sum())
    names = ["dq", "dk", "dv", "dg", "dbeta"] + ["dinitial_states"] * (h0 is not None)
    return dict(zip(names, torch.autograd.grad(loss, leaves, allow_unused=True)))


def norm(x, w=None, b=None, eps=1e-5, z=None):
    x = x.double()
    c = x - x.mean(-1, keepdim=True)
    y = c / (c.square().mean(-1, keepdim=True) + eps).sqrt()
    y = y * (1 if w is None else w.double()) + (0 if b is None else b.double())
    if z is not None:
        z = z.double()
        y = y * torch.where(z == -torch.inf, torch.zeros_like(z), z * torch.sigmoid(z))
    return y


def rel(a, ref):
    """2-norm of the difference over that of the reference (its own where that is 0)."""
    a, ref = a.double(), ref.double().to(a.device)
    n = ref.norm().item()
    return (a - ref).norm().item() / (n if n > 0 else 1.0)
