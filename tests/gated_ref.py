"""Plain 64-bit forms of the gated recurrence and its gradients, token by token, with bounds
on what 32-bit arithmetic may be off. Shared by the CPU and the GPU tests.

Bounds. With e = 2^-24 (half a unit in the last place of fp32, relative), each token of the
recurrence commits a few roundings: the gate and the write scale (ex2, a quotient, for tau != 1
two short series: at most 24 e relative), the product and sum (2 e), and, where runs of tokens
are joined, one rounding of the run's gate product per token and per join. An error made at
token t is carried on by the gates like the state itself. With
    M_t = |a_t| M_{t-1} + |a_t h_{t-1}| + |u_t|
the error of h_t is at most C e M_t, C = 64 covering the above with tau |log a| up to 4. The
adjoint has the same form. Outputs in 16 bits add half a step of theirs, eps/2 relative.
"""
import torch

E = 2.0 ** -24
C = 64 * E


def gates(z, gate, tau):
    if gate == "value":
        return z, 1 - z, torch.ones_like(z)
    w = tau * torch.nn.functional.logsigmoid(z)
    a = w.exp()
    return a, -torch.expm1(w), tau * a * torch.sigmoid(-z)


def scale(a, keep, write):
    """s and ds/da."""
    if write == "plain":
        return torch.ones_like(a), torch.zeros_like(a)
    if write == "leaky":
        return keep, -torch.ones_like(a)
    s = (keep * (1 + a)).clamp_min(0).sqrt()
    return s, torch.where(s > 0, -a / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))


def scan(x, z, h0, gate, write, tau, lengths=None, dy=None, dh_T=None):
    """Results and error bounds ("b_" names) in 64 bits; z [B,T,H] or [B,T,H,d]."""
    head = z.dim() == 3
    x, z = x.double(), z.double()
    B, T, H, d = x.shape
    zz = z.unsqueeze(-1).expand(x.shape) if head else z
    a, keep, da = gates(zz, gate, tau)
    s, ds = scale(a, keep, write)
    lens = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths]
    inside = torch.zeros((B, T, 1, 1), dtype=torch.bool, device=x.device)
    for b, v in enumerate(lens):
        inside[b, :v] = True
    zero, one = torch.zeros((), dtype=x.dtype, device=x.device), torch.ones((), dtype=x.dtype, device=x.device)
    a, s, x = torch.where(inside, a, one), torch.where(inside, s, zero), torch.where(inside, x, zero)
    u = s * x
    h = torch.zeros((B, H, d), dtype=x.dtype, device=x.device) if h0 is None else h0.double()
    m = torch.zeros_like(h)
    before, after, mag = [], [], []
    for t in range(T):
        before.append(h)
        m = a[:, t].abs() * m + (a[:, t] * h).abs() + u[:, t].abs()
        if lengths is not None:
            m = torch.where(inside[:, t], m, mag[-1] if mag else torch.zeros_like(m))
        h = a[:, t] * h + u[:, t]
        after.append(h)
        mag.append(m)
    st = lambda v: torch.stack(v, 1) if v else torch.zeros_like(x)  # noqa: E731
    y, hm = st(after), st(mag)
    out = {"y": torch.where(inside, y, zero), "h_T": h, "b_y": C * torch.where(inside, hm, zero), "b_h_T": C * m}
    if dy is None:
        return out
    dy = torch.where(inside, dy.double(), zero)
    k = torch.zeros_like(h) if dh_T is None else dh_T.double()
    km = torch.zeros_like(k)
    g, gm = [None] * T, [None] * T
    for t in range(T - 1, -1, -1):
        g[t] = dy[:, t] + k
        gm[t] = km + k.abs() + dy[:, t].abs()
        on = inside[:, t]
        k = a[:, t] * g[t]
        km = torch.where(on, a[:, t].abs() * gm[t] + k.abs(), km)
    out["dh0"], out["b_dh0"] = k, C * km
    g, gm, hp = st(g), st(gm), st(before)
    hpm = torch.cat([torch.zeros_like(hm[:, :1]), hm[:, :-1]], 1)
    out["dx"], out["b_dx"] = torch.where(inside, s * g, zero), C * torch.where(inside, s * gm, zero)
    part = torch.where(inside, g * da * (hp + x * ds), zero)
    size = hp.abs() + (x * ds).abs()
    bound = C * torch.where(inside, da.abs() * (gm * size + g.abs() * (hpm + size)), zero)
    if head:
        bound = bound.sum(-1) + d * E * part.abs().sum(-1)
        part = part.sum(-1)
    out["dz"], out["b_dz"] = part, bound
    return out


def check(got, want, name, rounded=None):
    """got is within the bound of want[name], plus half a step of got's type."""
    ref, bound = want[name], want["b_" + name]
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = 0.0 if got.dtype != torch.float16 else 2.0 ** -25  # fp16: half a step of its smallest numbers
    allowed = bound * (1 + half) + half * ref.abs() + tiny + 1e-37
    off = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), name
    worst = (off / allowed).max().item() if off.numel() else 0.0
    assert worst <= 1.0, (name, worst, off.max().item())
