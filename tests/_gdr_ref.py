"""Plain fp64 forms of the gated delta rule and of the norm and rotation of
queries and keys, on the CPU and differentiable: token by token, head by head
groups, straight from the definitions."""
import torch


def gdr(q, k, v, g, beta, S0, lens):
    """q, k [T, Hk, dk], v [T, Hv, dv], g, beta [T, Hv] (flat tokens), S0
    [N, Hv, dk, dv] or None; sequences of the given lengths one after another.
    Returns o [T, Hv, dv] and the last states, in fp64."""
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    o, states, t = [], [], 0
    for n, length in enumerate(lens):
        S = (torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64)
             if S0 is None else S0[n].double())
        for _ in range(length):
            S = torch.exp(g[t])[:, None, None] * S
            e = beta[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1))
            S = S + k[t][:, :, None] * e[:, None, :]
            o.append((q[t][:, :, None] * S).sum(1))
            t += 1
        states.append(S)
    out = torch.stack(o) if o else torch.zeros(0, v.shape[1], v.shape[2], dtype=torch.float64)
    return out, torch.stack(states)


def norm(x, kind, w=None, eps=1e-6):
    x = x.double()
    if kind == "rms":
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    elif kind == "l2":
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)
    return x if w is None else x * w.double()


def rotate(x, pos, freqs, layout, scale=1.0, inverse=False):
    """x [..., H, d] fp64, pos [...]; as complex numbers."""
    if freqs is None:
        return x
    rd = 2 * freqs.numel()
    a = pos.double()[..., None] * freqs.double()
    z = torch.polar(torch.full_like(a, scale), -a if inverse else a)[..., None, :]
    r = x[..., :rd]
    if layout == "half":
        z = torch.complex(r[..., :rd // 2], r[..., rd // 2:]) * z
        y = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.complex(r[..., 0::2], r[..., 1::2]) * z
        y = torch.stack([z.real, z.imag], -1).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def rel(got, ref):
    """2-norm of the difference over that of the reference; NaN anywhere fails."""
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    d = float((got - ref).norm())
    n = float(ref.norm())
    return d / n if n else d


def inputs(seed, lens, hk, hv, dk, dv, dtype, gate="slow", beta=1.0, s0=True):
    """Seeded inputs on the CPU in their own types, keys and queries unit rows."""
    r = torch.Generator().manual_seed(seed)
    t = sum(lens)

    def unit(*s):
        x = torch.randn(*s, generator=r, dtype=torch.float64)
        return x / x.norm(dim=-1, keepdim=True)

    q = (unit(t, hk, dk) * dk ** -0.5).to(dtype)
    k = unit(t, hk, dk).to(dtype)
    v = torch.randn(t, hv, dv, generator=r).to(dtype)
    g = -torch.rand(t, hv, generator=r)
    g = g * {"slow": 0.05, "fast": 20.0, "one": 0.0, "resets": 0.3}[gate]
    if gate == "resets":                 # a tenth of the tokens forget everything
        g = torch.where(torch.rand(t, hv, generator=r) < 0.1, -float("inf"), g)
    b = beta * torch.sigmoid(torch.randn(t, hv, generator=r))
    if t:
        b[t // 2] = 0.0                  # a token that writes nothing
    S0 = 0.3 * torch.randn(len(lens), hv, dk, dv, generator=r) if s0 else None
    return dict(q=q, k=k, v=v, g=g, beta=b, S0=S0)
