"""The block norms in 64 bits, with bounds on what 32-bit arithmetic may be off.

Bounds. With e = 2^-24, one row commits: a mean of squares of up to 16384 terms summed in
threads' runs of at most 32 and then pairwise (at most 32 + 14 roundings) and its reciprocal
square root (4 e), so at most 50 e relative on rho; the gate's activation and its derivative
16 e of their own size and of |gate| + 1 (gelu: formula 7.1.26 of Abramowitz and Stegun is
off by 7.5e-8 = 1.3 e in the distribution function; sigmoid: exp, a quotient); a few products.
Every result is a sum of products, so with T the same sum over absolute values, the error is at
most c T, c = 128 e, the terms of the means (another 46 e) included. Outputs in 16 bits add
half a step, eps/2 relative. Sums over N rows add N e of their absolute terms.
"""
import math

import torch

E = 2.0 ** -24
C = 128 * E


def act_of(g, act):
    """f, f', and what the arithmetic may be off in each, as a multiple of C."""
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
        f, df = g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        s = torch.sigmoid(g)
        f, df = (g * s, s * (1 + g * (1 - s))) if act == "silu" else (s, s * (1 - s))
    return f, df, (f.abs() + g.abs()) / 8, (df.abs() + g.abs() + 1) / 8


def forward(y, w_post, gate, act, residual, w_pre, pre, post, scale, eps):
    y = y.double()
    one = torch.ones(y.shape[-1], dtype=torch.float64, device=y.device)
    w = one if w_post is None else w_post.double()
    wp = one if w_pre is None else w_pre.double()
    rho1 = 1 / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() if post else torch.ones_like(y[..., :1])
    u = y * rho1
    f, df, bf, bdf = (torch.ones_like(y), torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(y)) if gate is None \
        else act_of(gate.double(), act)
    v = scale * u * w * f
    r = v if residual is None else residual.double() + v
    b_r = C * (v.abs() + (scale * u * w).abs() * bf + r.abs() / 32)
    out = {"r": r, "b_r": b_r}
    m = dict(y=y, w=w, wp=wp, rho1=rho1, u=u, f=f, df=df, bf=bf, bdf=bdf, r=r)
    if pre:
        rho2 = 1 / (r.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        out["n"] = r * rho2 * wp
        shift = (r.abs() * b_r).mean(-1, keepdim=True) * rho2.pow(2)
        out["b_n"] = (wp * rho2).abs() * (b_r + r.abs() * shift) + C * out["n"].abs()
        m.update(rho2=rho2)
    return out, m


def backward(y, w_post, gate, act, residual, w_pre, post, scale, eps, dr, dn):
    _, m = forward(y, w_post, gate, act, residual, w_pre, dn is not None, post, scale, eps)
    y, w, wp, rho1, u, f, df, r = (m[k] for k in ("y", "w", "wp", "rho1", "u", "f", "df", "r"))
    e = torch.zeros_like(y) if dr is None else dr.double()
    t = e.abs()
    out = {}
    if dn is not None:
        rho2, dn = m["rho2"], dn.double()
        e = e + rho2 * (wp * dn - r * rho2.pow(2) * (wp * dn * r).mean(-1, keepdim=True))
        # what the terms would be with nothing cancelling, r with the parts it is made of
        mag = r.abs() + (u * w * scale).abs() * (f.abs() + m["bf"]) + (0 if residual is None else residual.double().abs())
        t = t + rho2 * ((wp * dn).abs() + mag * rho2.pow(2) * (wp * dn * mag).abs().mean(-1, keepdim=True))
        rows = dn * r * rho2
        out["dw_pre"] = rows.flatten(0, -2).sum(0)
        out["b_dw_pre"] = (C * (dn * mag * rho2).abs() + rows.abs() * E * rows.flatten(0, -2).shape[0]).flatten(0, -2).sum(0)
    out["dresidual"], out["b_dresidual"] = e, C * t
    dv, tv = scale * e, abs(scale) * t
    out["dgate"] = dv * u * w * df
    out["b_dgate"] = C * (tv * (u * w).abs() * (df.abs() + m["bdf"]))
    rows = dv * u * f
    trows = tv * u.abs() * (f.abs() + m["bf"])
    out["dw_post"] = rows.flatten(0, -2).sum(0)
    out["b_dw_post"] = (C * trows + rows.abs() * E * rows.flatten(0, -2).shape[0]).flatten(0, -2).sum(0)
    du, tu = dv * w * f, tv * w.abs() * (f.abs() + m["bf"])
    if post:
        du = rho1 * (du - y * rho1.pow(2) * (du * y).mean(-1, keepdim=True))
        tu = rho1 * (tu + y.abs() * rho1.pow(2) * (tu * y.abs()).mean(-1, keepdim=True))
    out["dy"], out["b_dy"] = du, C * tu
    return out


def check(got, want, name):
    ref, bound = want[name], want["b_" + name]
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 1e-37
    allowed = bound * (1 + half) + half * ref.abs() + tiny
    off = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), name
    worst = (off / allowed).max().item() if off.numel() else 0.0
    assert worst <= 1.0, (name, worst, off.max().item())
