"""The operators around the SSD that are timed and compared with their plain forms.

Five operators: the gated delta rule over whole sequences (``delta_fwd``), its backward
(``delta_bwd``) and its single-token form (``delta_step``); the layer norm of the block's
output with the optional gate (``layer_norm``) and its backward (``layer_norm_bwd``).

Per batch row and head, with the group's q and k and a state S of headdim x dstate:

    S_t = exp(g_t) S_{t-1} + u_t k_t^T,   u_t = beta_t (v_t - exp(g_t) S_{t-1} k_t)
    y_t = scale S_t q_t

    y = ((x - mean(x)) rstd(x) w + b) SiLU(z)          over the last axis
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a short prompt in front of a decoder: latency
        dict(name="delta_fwd_prompt", op="delta_fwd", b=1, L=77, H=4, G=2, P=64, N=128, type="bf16", h0=True, seqs=0),
        # the benchmark's layer: one group of keys for 80 heads
        dict(name="delta_fwd_layer", op="delta_fwd", b=8, L=2048, H=80, G=1, P=64, N=128, type="bf16", h0=False, seqs=0),
        # a packed row of documents of 128 to 4096 tokens, wide value heads
        dict(name="delta_fwd_packed", op="delta_fwd", b=1, L=16384, H=32, G=8, P=128, N=128, type="bf16", h0=False,
             seqs=8),
        # 32-bit inputs, small heads, a length that no tile divides
        dict(name="delta_fwd_f32", op="delta_fwd", b=2, L=501, H=8, G=8, P=64, N=64, type="f32", h0=True, seqs=0),
        # a training step's backward
        dict(name="delta_bwd_layer", op="delta_bwd", b=4, L=2048, H=32, G=8, P=64, N=128, type="bf16", h0=False, seqs=0),
        # odd head sizes in 32 bits, a state handed in and its gradient out
        dict(name="delta_bwd_odd", op="delta_bwd", b=1, L=777, H=6, G=3, P=40, N=72, type="f32", h0=True, seqs=0),
        # one stream's decode step: latency
        dict(name="delta_step_one", op="delta_step", b=1, L=1, H=80, G=1, P=64, N=128, type="bf16", h0=True, seqs=0),
        # the decode step of 256 streams: the state does not fit the L2 cache
        dict(name="delta_step_many", op="delta_step", b=256, L=1, H=80, G=1, P=64, N=128, type="bf16", h0=True, seqs=0),
        # every head's output normalised over its headdim and gated
        dict(name="norm_heads_gated", op="layer_norm", rows=8 * 2048 * 80, D=64, type="bf16", affine=True, gate=True),
        # a decode step's rows at the model's inner width
        dict(name="norm_decode", op="layer_norm", rows=7, D=5120, type="bf16", affine=True, gate=False),
        # a training step's rows at the inner width, with the weight's and the bias's gradient
        dict(name="norm_bwd_wide", op="layer_norm_bwd", rows=16384, D=5120, type="bf16", affine=True, gate=False),
        # per-head rows with the gate, an odd width in 32 bits
        dict(name="norm_bwd_odd", op="layer_norm_bwd", rows=100003, D=129, type="f32", affine=True, gate=True),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_bwd", "delta_step", "layer_norm", "layer_norm_bwd"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("layer_norm", "layer_norm_bwd"):
        D = _log(rng, 4, 20000)
        rows = _log(rng, 1, max(1, (1 << 26) // D))
        return dict(op=op, rows=rows, D=D, type=kind, affine=rng.random() < 0.8, gate=rng.random() < 0.5)
    G = rng.choice([1, 1, 2, 3, 4, 8])
    H = G * rng.choice([1, 2, 3, 4, 8])
    P = rng.choice([16, 32, 64, 64, 128, _log(rng, 1, 256)])
    N = rng.choice([16, 64, 128, 128, _log(rng, 1, 256)])
    if op == "delta_step":
        N = (N + 3) // 4 * 4  # the step takes states in fours, as the SSD's does
        return dict(op=op, b=_log(rng, 1, max(1, min(512, (1 << 27) // (H * P * N)))), L=1, H=H, G=G, P=P, N=N,
                    type=kind, h0=True, seqs=0)
    most = (1 << 31) if op == "delta_fwd" else (1 << 29)  # values of the state over all tokens
    tokens = _log(rng, 1, max(1, min(16384, most // (H * P * N))))
    seqs = _log(rng, 1, 16) if rng.random() < 0.4 else 0
    if seqs:
        return dict(op=op, b=1, L=max(tokens, 2 * seqs), H=H, G=G, P=P, N=N, type=kind, h0=rng.random() < 0.3, seqs=seqs)
    b = min(tokens, _log(rng, 1, 8))
    return dict(op=op, b=b, L=max(1, min(4096, tokens // b)), H=H, G=G, P=P, N=N, type=kind, h0=rng.random() < 0.5, seqs=0)


# ------------------------------------------------------------------ the inputs
def _lengths(case, seed):
    """Tokens of each packed sequence: uneven, at least one each, from the seed."""
    n, L = case["seqs"], case["L"]
    gen = torch.Generator().manual_seed(seed)
    cut = (torch.randperm(L - 1, generator=gen)[: n - 1] + 1).sort().values.tolist()
    edge = [0] + cut + [L]
    return [edge[i + 1] - edge[i] for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    if case["op"] in ("layer_norm", "layer_norm_bwd"):
        rows, D = case["rows"], case["D"]
        s = dict(case=case, eps=1e-5, x=(normal(rows, D) * 1.5 + 0.3).to(t), weight=None, bias=None, z=None)
        if case["affine"]:
            s["weight"], s["bias"] = 1 + 0.2 * normal(D), 0.1 * normal(D)
        if case["gate"]:
            s["z"] = normal(rows, D).to(t)
        if case["op"] == "layer_norm_bwd":
            s["dy"] = normal(rows, D).to(t)
        return s
    b, L, H, G, P, N = (case[k] for k in ("b", "L", "H", "G", "P", "N"))
    unit = torch.nn.functional.normalize
    A = torch.exp(uniform(H) * math.log(16.0))
    dt = torch.exp(uniform(b, L, H) * math.log(100.0) + math.log(1e-3))
    s = dict(case=case, q=unit(normal(b, L, G, N), dim=-1).to(t), k=unit(normal(b, L, G, N), dim=-1).to(t),
             v=normal(b, L, H, P).to(t), g=-(dt * A), beta=torch.sigmoid(normal(b, L, H)), scale=N ** -0.5, h0=None,
             seq_idx=None, lengths=None)
    if case["h0"]:
        s["h0"] = 0.1 * normal(b, H, P, N)
    if case["seqs"]:
        s["lengths"] = _lengths(case, seed)
        ids = torch.repeat_interleave(torch.arange(case["seqs"]), torch.tensor(s["lengths"]))
        s["seq_idx"] = ids.to(torch.int32).reshape(1, L).to(DEV)
    if case["op"] == "delta_bwd":
        s["dy"] = normal(b, L, H, P).to(t)
        s["dfinal"] = 0.1 * normal(max(b, case["seqs"]), H, P, N)
    if case["op"] == "delta_step":
        for name in ("q", "k", "v", "g", "beta"):
            s[name] = s[name][:, 0].contiguous()
    return s


# ------------------------------------------------------------------ the plain forms
def _inverse(A):
    """(I + A)^-1 for strictly lower triangular A (..., C, C), blocks doubled from one to C."""
    C = A.shape[-1]
    T = torch.ones(*A.shape[:-2], C, 1, 1, device=A.device, dtype=A.dtype)
    size = 1
    while size < C:
        n = C // (2 * size)
        under = A.reshape(*A.shape[:-2], n, 2, size, n, 2, size)[..., 1, :, :, 0, :]
        under = under.diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        first, last = T[..., 0::2, :, :], T[..., 1::2, :, :]
        top = torch.cat([first, torch.zeros_like(first)], -1)
        T = torch.cat([top, torch.cat([-(last @ under @ first), last], -1)], -2)
        size *= 2
    return T[..., 0, :, :]


def _plain_delta(q, k, v, g, beta, scale, h0):
    """The delta rule chunk by chunk in 32 bits: (y, state after the last token)."""
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    R, nc = H // G, -(-L // CHUNK)
    pad = nc * CHUNK - L

    def chunks(t, heads, rest):
        t = torch.nn.functional.pad(t.float(), (0, 0) * (t.dim() - 2) + (0, pad))
        return t.reshape(b, nc, CHUNK, G, heads, *rest).movedim(2, 4)  # (b, nc, G, heads, C, ...)

    q, k, v = chunks(q, 1, (N,)), chunks(k, 1, (N,)), chunks(v, R, (P,))
    g, beta = chunks(g.unsqueeze(-1), R, (1,)).squeeze(-1), chunks(beta.unsqueeze(-1), R, (1,))
    cs = g.double().cumsum(-1)
    diff = (cs.unsqueeze(-1) - cs.unsqueeze(-2)).float()
    low = torch.ones(CHUNK, CHUNK, device=v.device, dtype=torch.bool).tril()
    decay = torch.where(low, diff, diff.new_tensor(-math.inf)).exp()
    kt = k.transpose(-1, -2)
    T = _inverse((beta * decay * (k @ kt)).tril(-1))
    M = scale * decay * (q @ kt)
    into = cs.float().exp().unsqueeze(-1)
    out_of = (cs[..., -1:] - cs).float().exp().unsqueeze(-1)
    whole = cs[..., -1].float().exp()[..., None, None]
    S = torch.zeros(b, G, R, P, N, device=v.device) if h0 is None else h0.reshape(b, G, R, P, N).float()
    ys = []
    for c in range(nc):
        St = S.transpose(-1, -2)
        u = T[:, c] @ (beta[:, c] * (v[:, c] - into[:, c] * (k[:, c] @ St)))
        ys.append(scale * into[:, c] * (q[:, c] @ St) + M[:, c] @ u)
        S = whole[:, c] * S + (out_of[:, c] * u).transpose(-1, -2) @ k[:, c]
    y = torch.stack(ys, 1).movedim(4, 2).reshape(b, nc * CHUNK, H, P)[:, :L]
    return y, S.reshape(b, H, P, N)


def _rows(t, lengths):
    """A packed row (1, L, ...) as one row for each sequence, zeros behind its end."""
    return torch.nn.utils.rnn.pad_sequence(list(t[0].split(lengths)), batch_first=True)


def _delta_of(s, q, k, v, g, beta, h0):
    """_plain_delta over the sequences of the state `s`, packed or not."""
    if s["lengths"] is None:
        return _plain_delta(q, k, v, g, beta, s["scale"], h0)
    n, most = s["lengths"], max(s["lengths"])
    if h0 is not None:  # the row's state enters its first sequence
        h0 = torch.cat([h0, h0.new_zeros(len(n) - 1, *h0.shape[1:])])
    y, fin = _plain_delta(*(_rows(t, n) for t in (q, k, v, g, beta)), s["scale"], h0)
    inside = torch.arange(most, device=y.device)[None] < torch.tensor(n, device=y.device)[:, None]
    return y[inside].unsqueeze(0), fin


def _plain_step(s):
    H, G = s["v"].shape[1], s["k"].shape[1]
    q, k = (s[n].float().repeat_interleave(H // G, 1).unsqueeze(2) for n in ("q", "k"))
    S = s["h0"] * s["g"].exp()[..., None, None]
    u = s["beta"].unsqueeze(-1) * (s["v"].float() - (S * k).sum(-1))
    S = S + u.unsqueeze(-1) * k
    s["h0"].copy_(S)
    return dict(y=(s["scale"] * (S * q).sum(-1)).to(s["v"].dtype), state=s["h0"])


def _normed(s):
    x = s["x"].float()
    c = x - x.mean(-1, keepdim=True)
    rstd = (c.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
    return c * rstd, rstd


def _plain_norm(s):
    y, _ = _normed(s)
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype)


def _plain_norm_bwd(s):
    n, rstd = _normed(s)
    t, dy, dz = s["x"].dtype, s["dy"].float(), None
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        full = n if s["weight"] is None else n * s["weight"] + s["bias"]
        dz = (dy * full * sig * (1 + z * (1 - sig))).to(t)
        dy = dy * z * sig
    dw = db = None
    if s["weight"] is not None:
        dw, db = (dy * n).sum(0, dtype=torch.float64).float(), dy.sum(0, dtype=torch.float64).float()
        dy = dy * s["weight"]
    dx = rstd * (dy - dy.mean(-1, keepdim=True) - n * (dy * n).mean(-1, keepdim=True))
    return dict(dx=dx.to(t), dweight=dw, dbias=db, dz=dz)


def _plain(s):
    op = s["case"]["op"]
    if op == "delta_step":
        return _plain_step(s)
    if op == "layer_norm":
        return _plain_norm(s)
    if op == "layer_norm_bwd":
        return _plain_norm_bwd(s)
    t = s["v"].dtype
    if op == "delta_fwd":
        y, fin = _delta_of(s, *(s[n] for n in ("q", "k", "v", "g", "beta", "h0")))
        return dict(y=y.to(t), final_states=fin)
    names = ["q", "k", "v", "g", "beta"] + ["h0"] * (s["h0"] is not None)
    leaves = [s[n].float().detach().requires_grad_() for n in names]
    y, fin = _delta_of(s, *leaves[:5], leaves[5] if s["h0"] is not None else None)
    grads = torch.autograd.grad([y, fin], leaves, [s["dy"].float(), s["dfinal"]])
    return {"d" + n: d.to(s[n].dtype) for n, d in zip(names, grads)}


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return _plain(s)
    import mamba_ssd_chunked_03_b200 as ssd

    op = s["case"]["op"]
    if op == "delta_fwd":
        y, fin = ssd.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], initial_states=s["h0"],
                               seq_idx=s["seq_idx"], num_seqs=s["case"]["seqs"] or None)
        return dict(y=y, final_states=fin)
    if op == "delta_bwd":
        d = ssd.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], scale=s["scale"],
                          initial_states=s["h0"], seq_idx=s["seq_idx"], num_seqs=s["case"]["seqs"] or None,
                          dfinal_states=s["dfinal"])
        got = {n: d[n] for n in ("dq", "dk", "dv", "dg", "dbeta")}
        if s["h0"] is not None:
            got["dh0"] = d["dinitial_states"]
        return got
    if op == "delta_step":
        y = ssd.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], scale=s["scale"])
        return dict(y=y, state=s["h0"])
    if op == "layer_norm":
        return ssd.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], z=s["z"])
    dx, dw, db, dz = ssd.layer_norm_bwd(s["x"], s["weight"], s["bias"], s["dy"], eps=s["eps"], z=s["z"])
    return dict(dx=dx, dweight=dw, dbias=db, dz=dz)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["type"] == "bf16" else 4
    if case["op"] in ("layer_norm", "layer_norm_bwd"):
        n, D = case["rows"] * case["D"], case["D"]
        back = case["op"] == "layer_norm_bwd"
        streams = (3 if back else 2) + (2 if back else 1) * case["gate"]
        return dict(bytes=n * e * streams + (4 if back else 2) * 4 * D * case["affine"],
                    flops=n * ((14 if back else 7) + (8 if back else 4) * case["gate"]))
    b, L, H, G, P, N = (case[k] for k in ("b", "L", "H", "G", "P", "N"))
    qk, v, gb = 2 * b * L * G * N * e, b * L * H * P * e, 2 * b * L * H * 4
    ends, h0 = max(b, case["seqs"]) * H * P * N * 4, b * H * P * N * 4 * case["h0"]
    if case["op"] == "delta_bwd":  # q, k, v, g, beta, dy, dfinal in; a gradient for each input out
        return dict(bytes=2 * (qk + v + gb) + v + ends + 2 * h0, flops=20 * b * L * H * P * N)
    return dict(bytes=qk + 2 * v + gb + ends + h0, flops=7 * b * L * H * P * N)


# ------------------------------------------------------------------ the definitions in 64 bits
def _tokens(s, H):
    """(t, rows, ...) views in 64 bits: one row for each sequence, zeros behind its end."""
    n = s["lengths"]
    got = []
    for name in ("q", "k", "v", "g", "beta"):
        t = s[name]
        if n is not None:
            t = _rows(t, n)
        t = t.double().transpose(0, 1)
        got.append(t.repeat_interleave(H // t.shape[2], 2) if name in ("q", "k") else t)
    return got


def _start(s, rows, H, P, N):
    S = torch.zeros(rows, H, P, N, device=DEV, dtype=torch.float64)
    if s["h0"] is not None:
        S[: s["h0"].shape[0]] = s["h0"].double()
    return S


def _mv(S, x):
    return (S @ x.unsqueeze(-1)).squeeze(-1)


def _outer(a, c):
    return a.unsqueeze(-1) * c.unsqueeze(-2)


def _ends(s, t, rows):
    """Which rows end with token t, or None when all end with the last one."""
    return None if s["lengths"] is None else torch.tensor([i for i in range(rows) if s["lengths"][i] == t + 1], device=DEV,
                                                           dtype=torch.long)


def _packed(s, y):
    """(t, rows, ...) back to the shape of the inputs."""
    y = y.transpose(0, 1)
    return y if s["lengths"] is None else torch.cat([y[i, :m] for i, m in enumerate(s["lengths"])]).unsqueeze(0)


def _exact_delta(s):
    _, L, H, P = s["v"].shape
    q, k, v, g, beta = _tokens(s, H)
    T, rows, N = q.shape[0], q.shape[1], q.shape[-1]
    S, fin, y = _start(s, rows, H, P, N), torch.zeros(rows, H, P, N, device=DEV, dtype=torch.float64), torch.empty_like(v)
    for t in range(T):
        S = S * g[t].exp()[..., None, None]
        S = S + _outer(beta[t].unsqueeze(-1) * (v[t] - _mv(S, k[t])), k[t])
        y[t] = s["scale"] * _mv(S, q[t])
        at = _ends(s, t, rows)
        if at is not None:
            fin[at] = S[at]
    return dict(y=_packed(s, y), final_states=S if s["lengths"] is None else fin)


def _exact_delta_bwd(s):
    _, L, H, P = s["v"].shape
    G = s["k"].shape[2]
    q, k, v, g, beta = _tokens(s, H)
    T, rows, N = q.shape[0], q.shape[1], q.shape[-1]
    if T * rows * H * P * N * 8 > 60e9 or T > 6000:
        return None
    dy = s["dy"] if s["lengths"] is None else _rows(s["dy"], s["lengths"])
    dy = s["scale"] * dy.double().transpose(0, 1)
    S = torch.empty(T + 1, rows, H, P, N, device=DEV, dtype=torch.float64)
    S[0] = _start(s, rows, H, P, N)
    for t in range(T):
        d = S[t] * g[t].exp()[..., None, None]
        S[t + 1] = d + _outer(beta[t].unsqueeze(-1) * (v[t] - _mv(d, k[t])), k[t])
    dq, dk, dv, dg, db = (torch.zeros_like(t) for t in (q, k, v, g, beta))
    A = s["dfinal"].double() if s["lengths"] is None else torch.zeros_like(S[0])
    for t in range(T - 1, -1, -1):  # A: the gradient of S_t from what comes after it
        at = _ends(s, t, rows)
        if at is not None:
            A[at] += s["dfinal"].double()[at]
        A = A + _outer(dy[t], q[t])
        dq[t] = _mv(S[t + 1].transpose(-1, -2), dy[t])
        D = S[t] * g[t].exp()[..., None, None]
        e = v[t] - _mv(D, k[t])
        du = _mv(A, k[t])
        db[t] = (du * e).sum(-1)
        de = beta[t].unsqueeze(-1) * du
        dv[t] = de
        dk[t] = _mv(A.transpose(-1, -2), beta[t].unsqueeze(-1) * e) - _mv(D.transpose(-1, -2), de)
        A = A - _outer(de, k[t])
        dg[t] = (A * D).sum((-1, -2))
        A = A * g[t].exp()[..., None, None]
    sums = [t.reshape(T, rows, G, H // G, N).sum(3) for t in (dq, dk)]
    got = dict(zip(("dq", "dk", "dv", "dg", "dbeta"), (_packed(s, t) for t in (*sums, dv, dg, db))))
    if s["h0"] is not None:
        got["dh0"] = A[: s["h0"].shape[0]]
    return got


def _exact_norm(s):
    x = s["x"].double().requires_grad_(s["case"]["op"] == "layer_norm_bwd")
    w, b, z = (None if s[n] is None else s[n].double().requires_grad_(x.requires_grad) for n in ("weight", "bias", "z"))
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    y = (x - mean) / (var + s["eps"]).sqrt()
    if w is not None:
        y = y * w + b
    if z is not None:
        y = y * z / (1 + (-z).exp())
    if not x.requires_grad:
        return y
    names = [n for n, t in (("dx", x), ("dweight", w), ("dbias", b), ("dz", z)) if t is not None]
    got = dict.fromkeys(("dx", "dweight", "dbias", "dz"))
    got.update(zip(names, torch.autograd.grad(y, [t for t in (x, w, b, z) if t is not None], s["dy"].double())))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("layer_norm", "layer_norm_bwd"):
        return _exact_norm(s)
    if op == "delta_bwd":
        return _exact_delta_bwd(s)
    if op == "delta_fwd":
        return _exact_delta(s) if max(s["lengths"] or [case["L"]]) <= 9000 else None
    for name in ("q", "k", "v", "g", "beta"):
        s[name] = s[name].unsqueeze(1)
    got = _exact_delta(s)
    return dict(y=got["y"][:, 0], state=got["final_states"])
