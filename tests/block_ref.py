"""64-bit forms of the short convolution, the selective scan and the layer norm, token by token, for the tests.

Every form is also run on magnitudes (mag=True: absolute values of the inputs that enter linearly), which bounds what
the terms of a sum can be; a kernel's rounding errors are counted against that."""
import torch


def close(got, want, mag, units, name):
    """got against want (64 bits): half a step of got's type, and `units` times 2^-24 of the magnitude of what was summed."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    value = got.double()
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + units * 2.0 ** -24 * mag
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # below 2^-14 its steps no longer shrink
    bad = ~((value - want).abs() <= tol)
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError((name, i, int(bad.sum()), float(value.flatten()[i]), float(want.flatten()[i]), float(tol.flatten()[i])))


def silu(v):
    return v * torch.sigmoid(v)


def silu_slope(v):
    s = torch.sigmoid(v)
    return s + v * s * (1 - s)


def clamp_lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths.tolist()]


def conv(x, w, bias=None, act="silu", state=None, lengths=None, dy=None, dstate_out=None):
    """({name: value}, {name: magnitude}) of the convolution and, with dy, of its gradients"""
    B, T, C = x.shape
    K = w.shape[1]
    w, b = w.double(), torch.zeros(C, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    out, mag = {}, {}
    names = ["y", "state"] + (["dx", "dstate", "dw", "dbias"] if dy is not None else [])
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=x.device)  # noqa: E731
    shapes = {"y": (B, T, C), "state": (B, K - 1, C), "dx": (B, T, C), "dstate": (B, K - 1, C), "dw": (C, K), "dbias": (C,)}
    for k in names:
        out[k], mag[k] = new(*shapes[k]), new(*shapes[k])
    for i, n in enumerate(clamp_lengths(lengths, B, T)):
        full = new(n + K - 1, C)
        if state is not None:
            full[:K - 1] = state[i].double()
        full[K - 1:] = x[i, :n].double()
        pre = b + sum(w[:, k] * full[k:k + n] for k in range(K))
        size = b.abs() + sum((w[:, k] * full[k:k + n]).abs() for k in range(K))
        out["y"][i, :n] = silu(pre) if act == "silu" else pre
        mag["y"][i, :n] = size
        out["state"][i] = full[n:]
        if dy is None:
            continue
        g = dy[i, :n].double()
        e = g * silu_slope(pre) if act == "silu" else g
        # the slope is at most 1.1 and changes by at most 0.5 per unit of pre
        me = g.abs() * (1.1 + 0.5 * size) if act == "silu" else g.abs()
        dfull, dmag = new(n + K - 1, C), new(n + K - 1, C)
        for k in range(K):
            dfull[k:k + n] += w[:, k] * e
            dmag[k:k + n] += w[:, k].abs() * me
        if dstate_out is not None:
            dfull[n:] += dstate_out[i].double()
            dmag[n:] += dstate_out[i].double().abs()
        out["dx"][i, :n], mag["dx"][i, :n] = dfull[K - 1:], dmag[K - 1:]
        out["dstate"][i], mag["dstate"][i] = dfull[:K - 1], dmag[:K - 1]
        out["dw"] += torch.stack([(e * full[k:k + n]).sum(0) for k in range(K)], 1)
        mag["dw"] += torch.stack([(me * full[k:k + n].abs()).sum(0) for k in range(K)], 1)
        out["dbias"] += e.sum(0)
        mag["dbias"] += me.sum(0)
    return out, mag


def selective(x, dt, A, b, c, skip=None, z=None, dt_bias=None, softplus=True, h0=None, lengths=None, dy=None, dh_T=None, mag=False):
    """{name: value} of the scan and, with dy, of its gradients; mag: of the magnitudes of their terms"""
    B, T, E = x.shape
    N = A.shape[1]
    f = (lambda t: t.double().abs()) if mag else (lambda t: t.double())  # noqa: E731
    if b.dim() == 3:
        b, c = b.unsqueeze(2), c.unsqueeze(2)
        flat = True
    else:
        flat = False
    G = b.shape[2]
    zero = lambda *s: torch.zeros(s, dtype=torch.float64, device=x.device)  # noqa: E731
    A = A.double()
    out = {"y": zero(B, T, E), "h_T": zero(B, E, N)}
    if dy is not None:
        out.update(dx=zero(B, T, E), ddt=zero(B, T, E), dA=zero(E, N), db=zero(B, T, G, N), dc=zero(B, T, G, N), dskip=zero(E),
                   dz=zero(B, T, E), ddt_bias=zero(E), dh0=zero(B, E, N))
    for i, n in enumerate(clamp_lengths(lengths, B, T)):
        raw = dt[i, :n].double() + (0 if dt_bias is None else dt_bias.double())
        d = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
        xs = f(x[i, :n])
        bs, cs = (f(t[i, :n]).repeat_interleave(E // G, dim=1) for t in (b, c))
        h = [zero(E, N) if h0 is None else f(h0[i])]
        for t in range(n):
            h.append(torch.exp(d[t][:, None] * A) * h[-1] + (d[t] * xs[t]).abs()[:, None] * bs[t] if mag else
                     torch.exp(d[t][:, None] * A) * h[-1] + (d[t] * xs[t])[:, None] * bs[t])
        out["h_T"][i] = h[-1]
        if n == 0:
            if dy is not None and dh_T is not None:
                out["dh0"][i] = f(dh_T[i])
            continue
        H = torch.stack(h)
        read = (H[1:] * cs).sum(-1)
        if skip is not None:
            read = read + f(skip) * xs
        gate = torch.ones_like(read) if z is None else silu(z[i, :n].double())
        gate = gate.abs() if mag else gate
        out["y"][i, :n] = read * gate
        if dy is None:
            continue
        g_y = f(dy[i, :n])
        if z is not None:
            # silu'(z) = s + z s (1 - s) with s = sigmoid(z): two terms, which cancel near z = -1.28
            zi = z[i, :n].double()
            s = torch.sigmoid(zi)
            out["dz"][i, :n] = g_y * read * (s + zi.abs() * s * (1 - s) if mag else silu_slope(zi))
        w = g_y * gate
        g = zero(E, N) if dh_T is None else f(dh_T[i])
        Aa = A.abs() if mag else A
        for t in range(n - 1, -1, -1):
            out["dc"][i, t] = (w[t][:, None] * H[t + 1]).reshape(G, E // G, N).sum(1)
            g = g + w[t][:, None] * cs[t]
            u = d[t] * xs[t]
            out["db"][i, t] = (g * u[:, None]).reshape(G, E // G, N).sum(1)
            du = (g * bs[t]).sum(-1)
            g = g * torch.exp(d[t][:, None] * A)
            q = g * H[t]
            out["dA"] += q * d[t][:, None]
            out["dx"][i, t] = d[t] * du + (0 if skip is None else f(skip) * w[t])
            dd = ((q * Aa).sum(-1) + du * xs[t]) * (torch.sigmoid(raw[t]) if softplus else 1.0)
            out["ddt"][i, t] = dd
            out["ddt_bias"] += dd
            if skip is not None:
                out["dskip"] += w[t] * xs[t]
        out["dh0"][i] = g
    if flat and dy is not None:
        out["db"], out["dc"] = out["db"][:, :, 0], out["dc"][:, :, 0]
    return out


def layer(x, w=None, b=None, residual=None, eps=1e-5, dn=None, dr=None):
    """({name: value}, {name: magnitude}) of the layer norm and, with dn, of its gradients"""
    out, mag = {}, {}
    r = x.double()
    if residual is not None:
        out["r"] = r + residual.double()
        mag["r"] = out["r"].abs()
        r = out["r"].to(residual.dtype).double()
    D = r.shape[-1]
    u = r - r.mean(-1, keepdim=True)
    var = (u * u).mean(-1, keepdim=True)
    rho = 1 / torch.sqrt(var + eps)
    # the mean is off by a few units of the row's mean magnitude, and with it every u, and rho of its row
    size = (u.abs() + r.abs().mean(-1, keepdim=True) + r.abs()) * rho
    W = torch.ones(D, dtype=torch.float64, device=r.device) if w is None else w.double()
    xhat = u * rho
    out["n"] = xhat * W + (0 if b is None else b.double())
    mag["n"] = size * W.abs() + (0 if b is None else b.double().abs())
    if dn is None:
        return out, mag
    g = dn.double()
    m = g * W
    out["dr"] = rho * (m - m.mean(-1, keepdim=True) - xhat * (m * xhat).mean(-1, keepdim=True))
    mag["dr"] = rho * (m.abs() + m.abs().mean(-1, keepdim=True) + size * (m.abs() * size).mean(-1, keepdim=True))
    if dr is not None:
        out["dr"] = out["dr"] + dr.double()
        mag["dr"] = mag["dr"] + dr.double().abs()
    lead = tuple(range(r.dim() - 1))
    out["dw"], mag["dw"] = (g * xhat).sum(lead), (g.abs() * size).sum(lead)
    out["db"], mag["db"] = g.sum(lead), g.abs().sum(lead)
    return out, mag
