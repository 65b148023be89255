"""Cases and plain forms of the operators around the state recurrence:

- "scan":  the gated linear recurrence h_t = a_t h_{t-1} + s(a_t) x_t over whole sequences,
- "train": the same with its backward pass (one training pass of the operator),
- "step":  the same for one token, on a batch of states,
- "norm":  the norm after a block with its gate and residual scale, joined with the norm before the next block,
- "normb": the backward pass of "norm".

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, with the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _scan_case(name, op, B, T, H, d, dtype, gate="logit", write="leaky", per="channel", zdtype=None, tau=1.0,
               fused=False, lengths=False, mean=3.0, std=1.0):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "d": d, "dtype": dtype, "gate": gate, "write": write,
            "per": per, "zdtype": zdtype or dtype, "tau": tau, "fused": fused, "lengths": lengths, "mean": mean, "std": std}


def _norm_case(name, op, N, D, dtype, ydtype=None, rdtype=None, wdtype="f32", post=True, gate="none", residual=True,
               pre=True, scale=1.0):
    return {"name": name, "op": op, "N": N, "D": D, "dtype": dtype, "ydtype": ydtype or dtype, "rdtype": rdtype or dtype,
            "wdtype": wdtype, "post": post, "gate": gate, "residual": residual, "pre": pre, "scale": scale}


def listed():
    return [
        # the small training shape; x and gate logits are the halves of one projection's output
        _scan_case("scan small training", "scan", 4, 2048, 8, 64, "bf16", fused=True),
        # the long-context shape: one sequence, few channels, long retention, norm-keeping writes
        _scan_case("scan long context", "scan", 1, 65536, 16, 128, "bf16", write="unit", tau=0.125, mean=4.0, std=0.5),
        # the mid-size layer with one forget gate per head and token, given as values in 32 bits
        _scan_case("scan head gates", "scan", 8, 4096, 16, 128, "bf16", gate="value", write="plain", per="head", zdtype="f32"),
        # forward and backward of the mid-size layer
        _scan_case("train mid layer", "train", 8, 4096, 16, 128, "bf16", fused=True),
        # a padded batch of ragged sequences in 32 bits with a gate per head
        _scan_case("train ragged heads", "train", 5, 1531, 3, 64, "f32", write="unit", per="head", lengths=True),
        # the decode batch: 256 sequences, one new token each
        _scan_case("step decode batch", "step", 256, 1, 32, 128, "bf16"),
        # one sequence, one token: latency
        _scan_case("step one sequence", "step", 1, 1, 16, 128, "bf16", write="unit"),
        # after the mid-size layer's output projection: norm, scaled residual in 32 bits, next block's norm
        _norm_case("norm mid layer", "norm", 8 * 4096, 16 * 128, "bf16", rdtype="f32", scale=0.5),
        # the mid-size layer's read-out (32 bits): per-head norm and GeLU gate
        _norm_case("norm read-out gate", "norm", 8 * 4096 * 16, 128, "bf16", ydtype="f32", gate="gelu", residual=False, pre=False),
        # the decode batch: 256 rows of 32 heads of 128
        _norm_case("norm decode batch", "norm", 256, 32 * 128, "bf16", wdtype="bf16", scale=0.25),
        # backward of the mid-size layer's norms
        _norm_case("normb mid layer", "normb", 8 * 4096, 16 * 128, "bf16", rdtype="f32", scale=0.5),
        # backward of the small training shape's read-out norm and gate
        _norm_case("normb read-out gate", "normb", 4 * 2048 * 8, 64, "bf16", ydtype="f32", gate="gelu", residual=False, pre=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm", "normb", "normb"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "normb"):
        D = rng.choice([_log_int(rng, 16, 16384), 8 * _log_int(rng, 2, 2048)])
        N = max(1, min(_log_int(rng, 1, 300000), (8 * 4096 * 16 * 128) // (2 * D)))
        gate = rng.choice(["none", "gelu", "silu", "sigmoid"])
        residual = rng.random() < 0.6
        c = _norm_case("", op, N, D, dtype, ydtype=rng.choice([dtype, "f32"]), rdtype=rng.choice([dtype, "f32"]) if residual else dtype,
                       wdtype=rng.choice([dtype, "f32"]), post=rng.random() < 0.8, gate=gate, residual=residual,
                       pre=rng.random() < 0.6, scale=rng.choice([1.0, 0.5, 0.125]))
    else:
        H = rng.randint(1, 32)
        per = rng.choice(["channel", "channel", "head"])
        d = rng.choice([16, 32, 64, 128]) if per == "head" or rng.random() < 0.6 else rng.randint(1, 160)
        B = _log_int(rng, 1, 512) if op == "step" else _log_int(rng, 1, 32)
        most = 8 * 4096 * 16 * 128 // 2
        T = 1 if op == "step" else max(1, min(_log_int(rng, 1, 65536), most // (B * H * d)))
        gate = rng.choice(["logit", "logit", "value"])
        zdtype = "f32" if gate == "value" else rng.choice([dtype, "f32"])
        c = _scan_case("", op, B, T, H, d, dtype, gate=gate, write=rng.choice(["plain", "leaky", "unit"]), per=per, zdtype=zdtype,
                       tau=rng.choice([1.0, 1.0, 0.125, 0.0625]) if gate == "logit" else 1.0,
                       fused=per == "channel" and zdtype == dtype and op != "step" and rng.random() < 0.5,
                       lengths=op != "step" and rng.random() < 0.4, mean=rng.choice([2.0, 3.0, 4.0]), std=rng.choice([0.5, 1.0]))
    del c["name"]
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    dt = DTYPES[c["dtype"]]
    if c["op"] in ("norm", "normb"):
        N, D = c["N"], c["D"]
        s = {"case": c, "y": normal(N, D, dtype=DTYPES[c["ydtype"]], std=0.7)}
        wt = DTYPES[c["wdtype"]]
        s["w_post"] = normal(D, mean=1.0, std=0.2, dtype=wt)
        s["w_pre"] = normal(D, mean=1.0, std=0.2, dtype=wt) if c["pre"] else None
        s["gate"] = normal(N, D, dtype=dt) if c["gate"] != "none" else None
        s["residual"] = normal(N, D, dtype=DTYPES[c["rdtype"]], std=2.0) if c["residual"] else None
        if c["op"] == "normb":
            s["dr"] = normal(N, D, dtype=DTYPES[c["rdtype"]] if c["residual"] else dt)
            s["dn"] = normal(N, D, dtype=dt) if c["pre"] else None
        return s
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    zt = DTYPES[c["zdtype"]]
    s = {"case": c, "h0": normal(B, H, d), "lengths": None}
    if c["op"] == "step":
        s["x"] = normal(B, H, d, dtype=dt)
        s["z"] = normal(*((B, H) if c["per"] == "head" else (B, H, d)), std=c["std"], mean=c["mean"])
        s["h_out"] = torch.empty_like(s["h0"])
    else:
        zshape = (B, T, H) if c["per"] == "head" else (B, T, H, d)
        if c["fused"]:  # x and z are slices of one projection's output
            both = torch.empty((B, T, 2, H, d), device="cuda", dtype=dt)
            both[:, :, 0] = normal(B, T, H, d, dtype=dt)
            both[:, :, 1] = normal(B, T, H, d, std=c["std"], mean=c["mean"], dtype=dt)
            s["x"], s["z"] = both[:, :, 0], both[:, :, 1]
        else:
            s["x"] = normal(B, T, H, d, dtype=dt)
            s["z"] = normal(*zshape, std=c["std"], mean=c["mean"])
    if c["gate"] == "value":
        s["z"] = torch.sigmoid(s["z"])
    if s["z"].dtype != zt:
        s["z"] = s["z"].to(zt)
    if c["op"] == "train":
        s["dy"] = normal(B, T, H, d, dtype=dt)
        s["dh_T"] = normal(B, H, d)
    if c["lengths"]:  # a padded batch: whatever stands behind a sequence's end is not to be used
        s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["lengths"][0] = T
        behind = torch.arange(T, device="cuda")[None] >= s["lengths"][:, None]
        s["x"][behind] = float("nan")
        s["z"][behind] = float("nan")
        if c["op"] == "train":
            s["dy"][behind] = float("nan")
    return s


# ---------------------------------------------------------------- plain forms

def _gates(z, c):
    """a, the write scale s(a), da/dz and ds/dz."""
    if c["gate"] == "value":
        a, da = z, torch.ones_like(z)
        keep, keep2 = 1 - a, (1 - a) * (1 + a)
    else:
        w = -c["tau"] * (torch.log1p(torch.exp(-z.abs())) + torch.relu(-z))
        a = torch.exp(w)
        keep, keep2 = -torch.expm1(w), -torch.expm1(2 * w)
        da = c["tau"] * a * torch.sigmoid(-z)
    if c["write"] == "plain":
        return a, torch.ones_like(a), da, torch.zeros_like(a)
    if c["write"] == "leaky":
        return a, keep, da, -da
    s = torch.sqrt(torch.relu(keep2))
    return a, s, da, torch.where(s > 0, -a * da / s, torch.zeros_like(s))


def _prefix(a, u):
    """All h_t = a_t h_{t-1} + u_t from h = 0: pairs of steps joined, the half-length recurrence, then the steps between."""
    T = u.shape[1]
    if T == 1:
        return u
    odd, even, end = a[:, 1::2], a[:, 0:T // 2 * 2:2], T // 2 * 2
    half = _prefix(odd * even, odd * u[:, 0:end:2] + u[:, 1::2])
    h = torch.empty_like(u)
    h[:, 1::2] = half
    h[:, :1] = u[:, :1]
    h[:, 2::2] = a[:, 2::2] * half[:, :(T - 1) // 2] + u[:, 2::2]
    return h


def _plain_scan(s, c):
    x, z = s["x"].float(), s["z"].float()
    z = z.unsqueeze(-1) if c["per"] == "head" else z
    a, w, da, dw = _gates(z, c)
    h0 = s["h0"].unsqueeze(1)
    if s["lengths"] is None:
        valid = None
    else:
        valid = (torch.arange(c["T"], device=x.device)[None] < s["lengths"][:, None])[:, :, None, None]
        zero = torch.zeros((), device=x.device)
        x, w, da, dw = (torch.where(valid, v, zero) for v in (x, w, da, dw))
        a = torch.where(valid, a, torch.ones((), device=x.device))
    u = w * x
    u[:, :1] += a[:, :1] * h0
    h = _prefix(a, u)
    y = h if valid is None else torch.where(valid, h, zero)
    out = {"y": y.to(s["x"].dtype), "h_T": h[:, -1].clone()}
    if c["op"] == "scan":
        return out
    dy = s["dy"].float()
    dy = dy.clone() if valid is None else torch.where(valid, dy, zero)
    dy[:, -1] += s["dh_T"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _prefix(after.flip(1), dy.flip(1)).flip(1)
    out["dh0"] = a[:, 0] * g[:, 0]
    h = torch.cat([h0, h[:, :-1]], 1)
    dz = g * (h * da + x * dw)
    out["dz"] = (dz.sum(-1) if c["per"] == "head" else dz).to(s["z"].dtype)
    out["dx"] = (g * w if valid is None else torch.where(valid, g * w, zero)).to(s["x"].dtype)
    return out


def _plain_step(s, c):
    z = s["z"].float()
    a, w, _, _ = _gates(z.unsqueeze(-1) if c["per"] == "head" else z, c)
    h = a * s["h0"] + w * s["x"].float()
    return {"h": h, "y": h.to(s["x"].dtype)}


def _act(g, kind):
    """The gate's activation and its derivative."""
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    p = torch.sigmoid(g)
    if kind == "silu":
        return g * p, p * (1 + g * (1 - p))
    return p, p * (1 - p)


EPS = 1e-6


def _plain_norm(s, c):
    y, w = s["y"].float(), s["w_post"].float()
    rho = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) if c["post"] else torch.ones((), device=y.device)
    u = y * rho
    f, df = (None, None) if c["gate"] == "none" else _act(s["gate"].float(), c["gate"])
    v = c["scale"] * u * w
    v = v if f is None else v * f
    r = v if s["residual"] is None else s["residual"].float() + v
    n, rho2 = None, None
    if c["pre"]:
        rho2 = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
        n = r * rho2 * s["w_pre"].float()
    if c["op"] == "norm":
        dt = DTYPES[c["dtype"]]
        out = {"r": r.to(DTYPES[c["rdtype"]] if c["residual"] else dt)}
        if n is not None:
            out["n"] = n.to(dt)
        return out
    e, out = s["dr"].float(), {}
    if c["pre"]:
        dn = s["dn"].float()
        out["dw_pre"] = (dn * r * rho2).sum(0)
        dn = dn * s["w_pre"].float()
        e = e + rho2 * (dn - r * rho2.square() * (dn * r).mean(-1, keepdim=True))
    if c["residual"]:
        out["dresidual"] = e.to(s["residual"].dtype)
    dv = c["scale"] * e
    if f is not None:
        out["dgate"] = (dv * u * w * df).to(s["gate"].dtype)
        dv = dv * f
    out["dw_post"] = (dv * u).sum(0)
    du = dv * w
    if c["post"]:
        du = rho * (du - u * (du * u).mean(-1, keepdim=True))
    out["dy"] = du.to(s["y"].dtype)
    return out


# ---------------------------------------------------------------- the library's operators

def _own_scan(L, s, c):
    how = {"gate": c["gate"], "write": c["write"], "tau": c["tau"], "lengths": s["lengths"]}
    if c["op"] == "scan":
        y, h_T = L.gated_scan_fwd(s["x"], s["z"], s["h0"], **how)
        return {"y": y, "h_T": h_T}
    marks = L.gated_scan_marks(s["x"])
    y, h_T = L.gated_scan_fwd(s["x"], s["z"], s["h0"], marks=marks, **how)
    grads = L.gated_scan_bwd(s["x"], s["z"], s["dy"], marks, dh_T=s["dh_T"], **how)
    return {"y": y, "h_T": h_T, "dx": grads["dx"], "dz": grads["dz"], "dh0": grads["dh0"]}


def _own_step(L, s, c):
    y = L.gated_step(s["h0"], s["x"], s["z"], gate=c["gate"], write=c["write"], tau=c["tau"], h_out=s["h_out"])
    return {"h": s["h_out"], "y": y}


def _own_norm(L, s, c):
    how = {"w_post": s["w_post"], "gate": s["gate"], "residual": s["residual"], "w_pre": s["w_pre"], "scale": c["scale"],
           "eps": EPS, "post_norm": c["post"]}
    if c["gate"] != "none":
        how["act"] = c["gate"]
    if c["op"] == "norm":
        r, n = L.block_norm_fwd(s["y"], out_dtype=DTYPES[c["dtype"]], **how)
        return {"r": r} if n is None else {"r": r, "n": n}
    grads = L.block_norm_bwd(s["y"], dr=s["dr"], dn=s["dn"], **how)
    return {k: v for k, v in grads.items() if v is not None}


def run(state):
    c = state["case"]
    kind = "norm" if c["op"] in ("norm", "normb") else "step" if c["op"] == "step" else "scan"
    if own:
        import orthogonal_update_recurrent_b200 as L
        return {"norm": _own_norm, "step": _own_step, "scan": _own_scan}[kind](L, state, c)
    return {"norm": _plain_norm, "step": _plain_step, "scan": _plain_scan}[kind](state, c)


# ---------------------------------------------------------------- work and the exact values

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    c = case
    if c["op"] in ("norm", "normb"):
        n, D = c["N"] * c["D"], c["D"]
        sx, sy, sr = _size(c["dtype"]), _size(c["ydtype"]), _size(c["rdtype"] if c["residual"] else c["dtype"])
        gate, res, pre = c["gate"] != "none", c["residual"], c["pre"]
        weights = D * _size(c["wdtype"]) * (2 if pre else 1)
        if c["op"] == "norm":
            per = sy + sx * gate + sr * res + sr + sx * pre
            return {"bytes": n * per + weights, "flops": n * (8 + 12 * gate + 5 * pre)}
        per = 2 * sy + 2 * sx * gate + 2 * sr * res + sr + sx * pre
        return {"bytes": n * per + weights + 4 * D * (2 if pre else 1), "flops": n * (16 + 20 * gate + 14 * pre)}
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    n, nz = B * T * H * d, B * T * H * (1 if c["per"] == "head" else d)
    sx, sz, state = _size(c["dtype"]), _size(c["zdtype"]), 4 * B * H * d
    if c["op"] == "train":
        return {"bytes": n * 4 * sx + nz * 2 * sz + 4 * state, "flops": 12 * n + 20 * nz}
    return {"bytes": n * 2 * sx + nz * sz + 2 * state, "flops": 4 * n + 8 * nz}


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    if c["op"] in ("norm", "normb"):
        return _exact_norm(s, c)
    x, z = s["x"].double(), s["z"].double()
    step = c["op"] == "step"
    if step:
        x, z = x.unsqueeze(1), z.unsqueeze(1)
    if c["per"] == "head":
        z = z[..., None].expand(x.shape)
    z = z.contiguous().requires_grad_(c["op"] == "train")
    if c["gate"] == "value":
        a = z * 1.0
        left = 1 - a
    else:
        log_a = c["tau"] * torch.nn.functional.logsigmoid(z)
        a, left = log_a.exp(), -torch.expm1(log_a)
    scale = {"plain": lambda: torch.ones_like(a), "leaky": lambda: left, "unit": lambda: (left * (1 + a)).clamp_min(0).sqrt()}[c["write"]]()
    B, T = x.shape[:2]
    lens = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    inside = torch.tensor([[t < n for t in range(T)] for n in lens], device=x.device)[:, :, None, None] if s["lengths"] is not None else None
    A, S = a.detach(), scale.detach()
    if inside is not None:
        x = x.masked_fill(~inside, 0.0)
        A, S = A.masked_fill(~inside, 1.0), S.masked_fill(~inside, 0.0)
    # time first, so that each step reads and writes whole blocks
    A, U = A.transpose(0, 1).contiguous(), (S * x).transpose(0, 1).contiguous()
    h = torch.empty((T + 1,) + tuple(U.shape[1:]), dtype=torch.float64, device=x.device)
    h[0] = s["h0"].double()
    for t in range(T):
        torch.addcmul(U[t], A[t], h[t], out=h[t + 1])
    y = h[1:].transpose(0, 1)
    if step:
        return {"h": y[:, 0].contiguous(), "y": y[:, 0].contiguous()}
    if inside is not None:
        y = y.masked_fill(~inside, 0.0)
    out = {"y": y.contiguous(), "h_T": h[T].clone()}
    if c["op"] == "scan":
        return out
    dy = s["dy"].double()
    dy = (dy if inside is None else dy.masked_fill(~inside, 0.0)).transpose(0, 1).contiguous()
    back = s["dh_T"].double()
    g = torch.empty_like(dy)
    for t in range(T - 1, -1, -1):
        torch.add(dy[t], back, out=g[t])
        back = A[t] * g[t]
    out["dh0"] = back
    g, before = g.transpose(0, 1), h[:T].transpose(0, 1)
    out["dx"] = (g * S).contiguous()
    ca, cs = g * before, g * x  # cotangents of a and of the write scale
    if inside is not None:
        ca, cs = ca.masked_fill(~inside, 0.0), cs.masked_fill(~inside, 0.0)
    dz, = torch.autograd.grad([a, scale] if scale.requires_grad else [a], z, [ca, cs] if scale.requires_grad else [ca])
    if inside is not None:
        dz = dz.masked_fill(~inside, 0.0)
    out["dz"] = dz.sum(-1) if c["per"] == "head" else dz
    return out


def _exact_norm(s, c):
    leaf = {k: s[k].double().requires_grad_(c["op"] == "normb") for k in ("y", "w_post", "gate", "residual", "w_pre") if s[k] is not None}
    b = leaf["y"]
    if c["post"]:
        b = b / (b.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt()
    b = b * leaf["w_post"] * c["scale"]
    if c["gate"] != "none":
        g = leaf["gate"]
        b = b * {"gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[c["gate"]](g)
    if c["residual"]:
        b = b + leaf["residual"]
    out = {"r": b}
    if c["pre"]:
        out["n"] = b / (b.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * leaf["w_pre"]
    if c["op"] == "norm":
        return out
    ends = [out["r"]] + ([out["n"]] if c["pre"] else [])
    starts = [s["dr"].double()] + ([s["dn"].double()] if c["pre"] else [])
    names = list(leaf)
    return {"d" + k: v for k, v in zip(names, torch.autograd.grad(ends, [leaf[k] for k in names], starts))}
