"""Cases and plain forms of the operators of a block with a selective state space:

- "conv":  the short causal convolution of every channel over whole sequences, with its activation,
- "convt": the same with its backward pass (one training pass of the operator),
- "convs": the same for one token,
- "scan":  the selective scan h_t = exp(dt_t A) h_{t-1} + dt_t x_t b_t, y_t = (c_t . h_t + skip x_t) silu(z_t) over whole sequences,
- "train": the same with its backward pass,
- "step":  the same for one token, on a batch of states,
- "ln":    the layer norm before a block, with the residual that it is added to,
- "lnt":   the same with its backward pass.

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, with the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def _conv_case(name, op, B, T, C, K, dtype, wdtype="f32", bias=True, act="silu", state=False, lengths=False, fused=False):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "K": K, "dtype": dtype, "wdtype": wdtype, "bias": bias, "act": act,
            "state": state, "lengths": lengths, "fused": fused}


def _scan_case(name, op, B, T, E, N, dtype, G=1, dtdtype=None, gate=True, skip=True, softplus=True, state=False, lengths=False,
               fused=False):
    return {"name": name, "op": op, "B": B, "T": T, "E": E, "N": N, "G": G, "dtype": dtype, "dtdtype": dtdtype or dtype,
            "gate": gate, "skip": skip, "softplus": softplus, "state": state, "lengths": lengths, "fused": fused}


def _norm_case(name, op, N, D, dtype, xdtype=None, rdtype=None, wdtype="f32", affine=True, residual=True):
    return {"name": name, "op": op, "N": N, "D": D, "dtype": dtype, "xdtype": xdtype or dtype, "rdtype": rdtype or dtype,
            "wdtype": wdtype, "affine": affine, "residual": residual}


def listed():
    return [
        # a prompt through the mid-size layer's convolution; x is a slice of the input projection's output
        _conv_case("conv mid layer", "conv", 8, 4096, 16 * 128, 4, "bf16", fused=True),
        # training on a padded batch of ragged sequences in 32 bits, three taps, a width that is no multiple of 8
        _conv_case("convt ragged", "convt", 5, 1531, 1026, 3, "f32", state=True, lengths=True),
        # the decode batch: 256 sequences, one new token each
        _conv_case("convs decode batch", "convs", 256, 1, 32 * 128, 4, "bf16", wdtype="bf16", state=True),
        # the small training shape, forward alone; x and z are the halves of one projection's output
        _scan_case("scan small training", "scan", 4, 2048, 8 * 64, 16, "bf16", fused=True),
        # the long-context shape: one sequence, continued from a state
        _scan_case("scan long context", "scan", 1, 65536, 16 * 64, 16, "bf16", state=True),
        # forward and backward of the mid-size layer
        _scan_case("train mid layer", "train", 8, 4096, 16 * 128, 16, "bf16", fused=True),
        # training on a padded batch of ragged sequences in 32 bits, two groups of b and c, an odd state size
        _scan_case("train ragged groups", "train", 5, 1531, 3 * 64, 13, "f32", G=2, gate=False, state=True, lengths=True),
        # the decode batch
        _scan_case("step decode batch", "step", 256, 1, 32 * 128, 16, "bf16", state=True),
        # one sequence, one token: latency
        _scan_case("step one sequence", "step", 1, 1, 16 * 128, 16, "bf16", state=True),
        # before the mid-size layer's block: the block's output added to a residual stream in 32 bits, and its norm
        _norm_case("ln mid layer", "ln", 8 * 4096, 16 * 128, "bf16", rdtype="f32"),
        # the decode batch: 256 rows of 32 heads of 128
        _norm_case("ln decode batch", "ln", 256, 32 * 128, "bf16", wdtype="bf16"),
        # one training pass of the mid-size layer's norm
        _norm_case("lnt mid layer", "lnt", 8 * 4096, 16 * 128, "bf16", rdtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "convt", "convt", "convs", "scan", "scan", "train", "train", "step", "ln", "lnt", "lnt"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("ln", "lnt"):
        D = rng.choice([_log_int(rng, 16, 16384), 8 * _log_int(rng, 2, 2048)])
        N = max(1, min(_log_int(rng, 1, 300000), (8 * 4096 * 16 * 128) // (2 * D)))
        residual = rng.random() < 0.6
        c = _norm_case("", op, N, D, dtype, xdtype=rng.choice([dtype, "f32"]) if residual else dtype,
                       rdtype=rng.choice([dtype, "f32"]), wdtype=rng.choice([dtype, "f32"]), affine=rng.random() < 0.85, residual=residual)
        if not residual:
            c["rdtype"] = c["xdtype"]
    elif op in ("conv", "convt", "convs"):
        C = rng.choice([_log_int(rng, 1, 8192), 8 * _log_int(rng, 2, 1024)])
        B = _log_int(rng, 1, 512) if op == "convs" else _log_int(rng, 1, 32)
        T = 1 if op == "convs" else max(1, min(_log_int(rng, 1, 65536), 8 * 4096 * 16 * 128 // (2 * B * C)))
        c = _conv_case("", op, B, T, C, rng.choice([2, 3, 4, 4, 4, 5, 7, 8]), dtype, wdtype=rng.choice([dtype, "f32"]),
                       bias=rng.random() < 0.8, act=rng.choice(["silu", "silu", "none"]), state=op == "convs" or rng.random() < 0.4,
                       lengths=op != "convs" and rng.random() < 0.4, fused=op != "convs" and rng.random() < 0.4)
    else:
        N = rng.choice([16, 16, 16, 8, 32, 64, 128, rng.randint(1, 40)])
        G = rng.choice([1, 1, 1, 2, 4])
        E = G * rng.choice([_log_int(rng, 8, 1024), 8 * _log_int(rng, 2, 128)])
        B = _log_int(rng, 1, 512) if op == "step" else _log_int(rng, 1, 32)
        T = 1 if op == "step" else max(1, min(_log_int(rng, 1, 65536), 8 * 4096 * 16 * 128 * 16 // (4 * B * E * max(N, 4))))
        softplus = rng.random() < 0.8
        c = _scan_case("", op, B, T, E, N, dtype, G=G, dtdtype=rng.choice([dtype, "f32"]) if softplus else "f32",
                       gate=rng.random() < 0.7, skip=rng.random() < 0.8, softplus=softplus, state=op == "step" or rng.random() < 0.5,
                       lengths=op != "step" and rng.random() < 0.4, fused=op != "step" and rng.random() < 0.3)
    del c["name"]
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    def slices(n, *shape):
        """n tensors of x's type, with c["fused"] slices of one projection's output"""
        if not c["fused"]:
            return [normal(*shape, dtype=dt) for _ in range(n)]
        wide = normal(*shape[:-1], 2, shape[-1], dtype=dt)
        return [wide[..., k, :] for k in range(n)]

    s = {"case": c, "lengths": None}
    if c["op"] in ("ln", "lnt"):
        N, D = c["N"], c["D"]
        s["x"] = normal(N, D, dtype=DTYPES[c["xdtype"]], mean=0.1)
        s["residual"] = normal(N, D, dtype=DTYPES[c["rdtype"]], std=2.0, mean=0.3) if c["residual"] else None
        s["w"] = normal(D, mean=1.0, std=0.2, dtype=DTYPES[c["wdtype"]]) if c["affine"] else None
        s["b"] = normal(D, std=0.2, dtype=DTYPES[c["wdtype"]]) if c["affine"] else None
        if c["op"] == "lnt":
            s["dn"] = normal(N, D, dtype=dt)
            s["dr"] = normal(N, D, dtype=DTYPES[c["rdtype"]]) if c["residual"] else None
        return s
    B, T = c["B"], c["T"]
    tokens = (B,) if c["op"] in ("convs", "step") else (B, T)
    if c["op"] in ("conv", "convt", "convs"):
        C, K = c["C"], c["K"]
        s["x"], = slices(1, *tokens, C)
        s["w"] = normal(C, K, std=K ** -0.5, dtype=DTYPES[c["wdtype"]])
        s["bias"] = normal(C, std=0.2, dtype=DTYPES[c["wdtype"]]) if c["bias"] else None
        s["state"] = normal(B, K - 1, C, dtype=dt) if c["state"] else None
        if c["op"] == "convs":
            s["state_out"] = torch.empty_like(s["state"])
        if c["op"] == "convt":
            s["dy"] = normal(B, T, C, dtype=dt)
            s["dstate"] = normal(B, K - 1, C, dtype=dt) if c["state"] else None
        behind = ("x", "dy")
    else:
        E, N, G = c["E"], c["N"], c["G"]
        if c["gate"]:
            s["x"], s["z"] = slices(2, *tokens, E)
        else:
            (s["x"],), s["z"] = slices(1, *tokens, E), None
        s["b"] = normal(*tokens, G, N, dtype=dt)
        s["c"] = normal(*tokens, G, N, dtype=dt)
        s["A"] = -torch.arange(1, N + 1, device="cuda").float() * torch.exp(normal(E, N, std=0.1))
        s["skip"] = normal(E, mean=1.0, std=0.1) if c["skip"] else None
        # steps between 1/1000 and 1/10
        first = torch.exp(torch.rand((E,), generator=gen, device="cuda") * math.log(100.0) + math.log(0.001))
        s["dt_bias"] = torch.log(torch.expm1(first)) if c["softplus"] else None
        s["dt"] = normal(*tokens, E, std=0.5, dtype=DTYPES[c["dtdtype"]])
        if not c["softplus"]:
            s["dt"] = (s["dt"].exp() * first).to(s["dt"].dtype)
        s["h0"] = normal(B, E, N) if c["state"] else None
        if c["op"] == "step":
            s["h_out"] = torch.empty_like(s["h0"])
        if c["op"] == "train":
            s["dy"] = normal(B, T, E, dtype=dt)
            s["dh_T"] = normal(B, E, N) if c["state"] else None
        behind = ("x", "z", "dt", "b", "c", "dy")
    if c["lengths"]:  # a padded batch: whatever stands behind a sequence's end is not to be used
        s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["lengths"][0] = T
        pad = torch.arange(T, device="cuda")[None] >= s["lengths"][:, None]
        for k in behind:
            if s.get(k) is not None:
                s[k][pad] = float("nan")
    return s


# ---------------------------------------------------------------- plain forms

def _inside(s, T, like):
    """[B, T, 1...] whether a token stands before its sequence's end, or None"""
    if s["lengths"] is None:
        return None
    m = torch.arange(T, device=like.device)[None] < s["lengths"][:, None]
    return m.reshape(m.shape + (1,) * (like.dim() - 2))


def _cut(t, inside):
    """t in 32 bits, 0 behind a sequence's end"""
    t = t.float()
    return t if inside is None else torch.where(inside, t, torch.zeros((), device=t.device))


def _plain_conv(s, c):
    K, T, dt = c["K"], c["T"], s["x"].dtype
    step = c["op"] == "convs"
    x = s["x"].unsqueeze(1) if step else s["x"]
    B, C = x.shape[0], x.shape[2]
    inside = _inside(s, T, x)
    before = torch.zeros((B, K - 1, C), device=x.device) if s["state"] is None else s["state"].float()
    full = torch.cat([before, _cut(x, inside)], 1)
    w = s["w"].float()
    pre = sum(w[:, k] * full[:, k:k + T] for k in range(K))
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    sig = torch.sigmoid(pre) if c["act"] == "silu" else None
    y = _cut(pre if sig is None else pre * sig, inside).to(dt)
    if s["lengths"] is None:
        state = full[:, T:].to(dt)
    else:
        ends = s["lengths"].long()[:, None] + torch.arange(K - 1, device=x.device)
        state = torch.gather(full, 1, ends[:, :, None].expand(-1, -1, C)).to(dt)
    if step:
        return {"y": y[:, 0], "state": state}
    out = {"y": y, "state": state}
    if c["op"] == "conv":
        return out
    dpre = _cut(s["dy"], inside)
    if sig is not None:
        dpre = dpre * sig * (1 + pre * (1 - sig))
    dpre = _cut(dpre, inside)
    late = torch.cat([torch.zeros_like(before), dpre, torch.zeros_like(before)], 1)
    dfull = sum(w[:, K - 1 - j] * late[:, j:j + T + K - 1] for j in range(K))
    if s["dstate"] is not None:
        ds = s["dstate"].float()
        if s["lengths"] is None:
            dfull[:, T:] += ds
        else:
            dfull.scatter_add_(1, ends[:, :, None].expand(-1, -1, C), ds)
    out["dx"] = _cut(dfull[:, K - 1:], inside).to(dt)
    if s["state"] is not None:
        out["dstate"] = dfull[:, :K - 1].to(dt)
    out["dw"] = torch.stack([(dpre * full[:, k:k + T]).sum((0, 1)) for k in range(K)], 1)
    if s["bias"] is not None:
        out["dbias"] = dpre.sum((0, 1))
    return out


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


def _spread(t, E):
    """[B, T, G, N] to every channel of its group, [B, T, E, N]"""
    B, T, G, N = t.shape
    return t[:, :, :, None].expand(B, T, G, E // G, N).reshape(B, T, E, N)


def _gather(t, G):
    """[B, T, E, N] summed over every group's channels"""
    B, T, E, N = t.shape
    return t.reshape(B, T, G, E // G, N).sum(3)


def _plain_scan(s, c):
    step, E, G = c["op"] == "step", c["E"], c["G"]
    names = ("x", "z", "dt", "b", "c")
    t = {k: s[k].unsqueeze(1) if step and s[k] is not None else s[k] for k in names}
    inside = _inside(s, c["T"], t["x"])
    raw = t["dt"].float() if s["dt_bias"] is None else t["dt"].float() + s["dt_bias"]
    raw = _cut(raw, inside)
    dt = torch.relu(raw) + torch.log1p(torch.exp(-raw.abs())) if c["softplus"] else raw
    dt = _cut(dt, inside)
    x = _cut(t["x"], inside)
    wide = None if inside is None else inside[..., None]
    b, cc = _spread(_cut(t["b"], wide), E), _spread(_cut(t["c"], wide), E)
    a = torch.exp(dt[..., None] * s["A"])
    u = (dt * x)[..., None] * b
    if s["h0"] is not None:
        u[:, 0] += a[:, 0] * s["h0"]
    h = _prefix(a, u)
    read = (h * cc).sum(-1)
    if s["skip"] is not None:
        read = read + s["skip"] * x
    if s["z"] is not None:
        z = _cut(t["z"], inside)
        sig = torch.sigmoid(z)
    y = read if s["z"] is None else read * z * sig
    y = _cut(y, inside).to(s["x"].dtype)
    if step:
        return {"y": y[:, 0], "h": h[:, 0]}
    out = {"y": y, "h_T": h[:, -1].clone()}
    if c["op"] == "scan":
        return out
    dread = _cut(s["dy"], inside)
    if s["z"] is not None:
        out["dz"] = (dread * read * sig * (1 + z * (1 - sig))).to(s["x"].dtype)
        dread = dread * z * sig
    out["dc"] = _gather(dread[..., None] * h, G).to(s["x"].dtype)
    g = dread[..., None] * cc
    if s["dh_T"] is not None:
        g[:, -1] += s["dh_T"]
    g = _prefix(torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1), g.flip(1)).flip(1)
    du = (g * b).sum(-1)
    out["db"] = _gather(g * (dt * x)[..., None], G).to(s["x"].dtype)
    dx = du * dt
    if s["skip"] is not None:
        dx = dx + s["skip"] * dread
        out["dskip"] = (dread * x).sum((0, 1))
    out["dx"] = _cut(dx, inside).to(s["x"].dtype)
    g *= a
    if s["h0"] is not None:
        out["dh0"] = g[:, 0].clone()
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    g *= torch.cat([first, h[:, :-1]], 1)
    out["dA"] = (g * dt[..., None]).sum((0, 1))
    ddt = (g * s["A"]).sum(-1) + du * x
    if c["softplus"]:
        ddt = ddt * torch.sigmoid(raw)
    ddt = _cut(ddt, inside)
    out["ddt"] = ddt.to(s["dt"].dtype)
    if s["dt_bias"] is not None:
        out["ddt_bias"] = ddt.sum((0, 1))
    return out


def _plain_norm(s, c):
    r = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["r"] = (r + s["residual"].float()).to(s["residual"].dtype)
        r = out["r"].float()
    u = r - r.mean(-1, keepdim=True)
    rho = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    u = u * rho
    n = u if s["w"] is None else u * s["w"].float() + s["b"].float()
    out["n"] = n.to(DTYPES[c["dtype"]])
    if c["op"] == "ln":
        return out
    dn = s["dn"].float()
    du = dn if s["w"] is None else dn * s["w"].float()
    dr = rho * (du - du.mean(-1, keepdim=True) - u * (du * u).mean(-1, keepdim=True))
    if s["dr"] is not None:
        dr = dr + s["dr"].float()
    out["dr"] = dr.to(DTYPES[c["rdtype"]])
    if c["xdtype"] != c["rdtype"]:
        out["dx"] = dr.to(s["x"].dtype)
    if s["w"] is not None:
        out["dw"], out["db"] = (dn * u).sum(0), dn.sum(0)
    return out


# ---------------------------------------------------------------- the library's operators

def _own_conv(L, s, c):
    how = {"bias": s["bias"], "act": c["act"]}
    if c["op"] == "convs":
        y = L.short_conv_step(s["state"], s["x"], s["w"], state_out=s["state_out"], **how)
        return {"y": y, "state": s["state_out"]}
    how.update(state=s["state"], lengths=s["lengths"])
    y, state = L.short_conv_fwd(s["x"], s["w"], **how)
    out = {"y": y, "state": state}
    if c["op"] == "convt":
        out.update(L.short_conv_bwd(s["x"], s["w"], s["dy"], dstate_out=s["dstate"], **how))
    return {k: v for k, v in out.items() if v is not None}


def _own_scan(L, s, c):
    how = {"z": s["z"], "dt_bias": s["dt_bias"], "softplus": c["softplus"]}
    tensors = (s["x"], s["dt"], s["A"], s["b"], s["c"])
    if c["op"] == "step":
        y = L.selective_step(s["h0"], *tensors, s["skip"], h_out=s["h_out"], **how)
        return {"y": y, "h": s["h_out"]}
    how["lengths"] = s["lengths"]
    if c["op"] == "scan":
        y, h_T = L.selective_scan_fwd(*tensors, s["skip"], h0=s["h0"], **how)
        return {"y": y, "h_T": h_T}
    marks = L.selective_scan_marks(s["x"], c["N"])
    y, h_T = L.selective_scan_fwd(*tensors, s["skip"], h0=s["h0"], marks=marks, **how)
    grads = L.selective_scan_bwd(*tensors, s["dy"], marks, s["skip"], dh_T=s["dh_T"], **how)
    if s["h0"] is None:
        del grads["dh0"]
    return {"y": y, "h_T": h_T, **{k: v for k, v in grads.items() if v is not None}}


def _own_norm(L, s, c):
    r, n = L.layer_norm_fwd(s["x"], s["w"], s["b"], residual=s["residual"], eps=EPS, out_dtype=DTYPES[c["dtype"]])
    out = {"n": n} if s["residual"] is None else {"r": r, "n": n}
    if c["op"] == "lnt":
        grads = L.layer_norm_bwd(r, s["dn"], s["w"], s["b"], dr=s["dr"], eps=EPS, x_dtype=s["x"].dtype)
        if c["xdtype"] == c["rdtype"]:
            del grads["dx"]  # it is dr
        out.update((k, v) for k, v in grads.items() if v is not None)
    return out


def run(state):
    c = state["case"]
    kind = "norm" if c["op"] in ("ln", "lnt") else "conv" if c["op"] in ("conv", "convt", "convs") else "scan"
    if own:
        import orthogonal_update_recurrent_b200 as L
        return {"norm": _own_norm, "conv": _own_conv, "scan": _own_scan}[kind](L, state, c)
    return {"norm": _plain_norm, "conv": _plain_conv, "scan": _plain_scan}[kind](state, c)


# ---------------------------------------------------------------- work and the exact values

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    c = case
    sx = _size(c["dtype"])
    if c["op"] in ("ln", "lnt"):
        n, D, res = c["N"] * c["D"], c["D"], c["residual"]
        si, sr = _size(c["xdtype"]), _size(c["rdtype"])
        weights = 2 * D * _size(c["wdtype"]) if c["affine"] else 0
        per, flops = si + 2 * sr * res + sx, 9 * n
        if c["op"] == "lnt":  # r, dn and dr read again, dr and dx written
            per += (sr if res else si) + sx + sr * res + sr + (si if si != sr else 0)
            weights += 8 * D if c["affine"] else 0
            flops += 15 * n
        return {"bytes": n * per + weights, "flops": flops}
    if c["op"] in ("conv", "convt", "convs"):
        n, K = c["B"] * c["T"] * c["C"], c["K"]
        act = 4 if c["act"] == "silu" else 0
        state = c["B"] * (K - 1) * c["C"] * sx
        weights = c["C"] * (K * _size(c["wdtype"]) + (_size(c["wdtype"]) if c["bias"] else 0))
        total = {"bytes": 2 * n * sx + state * (2 if c["state"] else 1) + weights, "flops": n * (2 * K + act)}
        if c["op"] == "convt":
            total["bytes"] += 3 * n * sx + 2 * state * c["state"] + 4 * c["C"] * (K + c["bias"])
            total["flops"] += n * (6 * K + 2 * act)
        return total
    n, N, G = c["B"] * c["T"] * c["E"], c["N"], c["G"]
    sd, gate = _size(c["dtdtype"]), c["gate"]
    bc, state = 2 * c["B"] * c["T"] * G * N * sx, 4 * c["B"] * c["E"] * N
    weights = 4 * c["E"] * (N + c["skip"] + c["softplus"])
    total = {"bytes": n * (sx * (2 + gate) + sd) + bc + state * (2 if c["state"] else 1) + weights,
             "flops": n * (6 * N + 10 + 4 * gate)}
    if c["op"] == "train":
        total["bytes"] += n * (sx * (3 + 2 * gate) + 2 * sd) + 2 * bc + 2 * state * c["state"] + weights
        total["flops"] += n * (20 * N + 20 + 8 * gate)
    return total


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    if c["op"] in ("ln", "lnt"):
        return _exact_norm(s, c)
    if c["op"] in ("conv", "convt", "convs"):
        return _exact_conv(s, c)
    return _exact_scan(s, c)


def _mask(s, c):
    """[B, T] in 64 bits, 1 before a sequence's end"""
    if s["lengths"] is None:
        return torch.ones((c["B"], c["T"]), dtype=torch.float64, device="cuda")
    return torch.tensor([[float(t < n) for t in range(c["T"])] for n in s["lengths"].tolist()], dtype=torch.float64, device="cuda")


def _exact_conv(s, c):
    K, T, train = c["K"], c["T"], c["op"] == "convt"
    m = _mask(s, c)[:, :, None]
    x = s["x"].unsqueeze(1) if c["op"] == "convs" else s["x"]
    x = x.double().masked_fill(m == 0, 0.0).requires_grad_(train)
    w = s["w"].double().requires_grad_(train)
    bias = None if s["bias"] is None else s["bias"].double().requires_grad_(train)
    state = None if s["state"] is None else s["state"].double().requires_grad_(train)
    seq = torch.nn.functional.pad(x, (0, 0, K - 1, 0)) if state is None else torch.cat([state, x], 1)
    y = torch.nn.functional.conv1d(seq.transpose(1, 2), w[:, None, :], bias, groups=c["C"]).transpose(1, 2)
    y = (torch.nn.functional.silu(y) if c["act"] == "silu" else y) * m
    lens = [T] * c["B"] if s["lengths"] is None else s["lengths"].tolist()
    last = torch.stack([seq[i, n:n + K - 1] for i, n in enumerate(lens)])
    if c["op"] == "convs":
        return {"y": y[:, 0], "state": last}
    out = {"y": y.detach(), "state": last.detach()}
    if not train:
        return out
    loss = (y * s["dy"].double().masked_fill(m == 0, 0.0)).sum()
    if s["dstate"] is not None:
        loss = loss + (last * s["dstate"].double()).sum()
    names = [k for k, v in (("dx", x), ("dw", w), ("dbias", bias), ("dstate", state)) if v is not None]
    grads = torch.autograd.grad(loss, [{"dx": x, "dw": w, "dbias": bias, "dstate": state}[k] for k in names])
    out.update(zip(names, grads))
    out["dx"] = out["dx"] * m
    return out


def _exact_scan(s, c):
    step, train = c["op"] == "step", c["op"] == "train"
    B, T, E, N, G = c["B"], c["T"], c["E"], c["N"], c["G"]
    m = _mask(s, c)

    def wide(t):  # time first, 0 behind the end
        t = t.unsqueeze(1) if step else t
        t = t.double().masked_fill(m.reshape(m.shape + (1,) * (t.dim() - 2)) == 0, 0.0)
        return t.transpose(0, 1).contiguous()

    x, dt, b, cc = (wide(s[k]) for k in ("x", "dt", "b", "c"))
    mt = m.t()[:, :, None]
    raw = dt if s["dt_bias"] is None else dt + s["dt_bias"].double()
    delta = (torch.logaddexp(raw, torch.zeros_like(raw)) if c["softplus"] else raw) * mt
    A = s["A"].double()
    h = torch.zeros((T + 1 if train else 2, B, E, N), dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h[0] = s["h0"].double()
    read = torch.empty((T, B, E), dtype=torch.float64, device="cuda")
    v = delta * x

    def at(t, i):  # [B, E, N] of a token's groups
        return t[i].repeat_interleave(E // G, dim=1)

    for i in range(T):
        now, nxt = (i, i + 1) if train else (i % 2, (i + 1) % 2)
        torch.addcmul((delta[i][..., None] * A).exp_().mul_(h[now]), v[i][..., None], at(b, i), out=h[nxt])
        torch.sum(h[nxt] * at(cc, i), -1, out=read[i])
    if s["skip"] is not None:
        read += s["skip"].double() * x
    z = None if s["z"] is None else wide(s["z"])
    y = (read if z is None else read * torch.nn.functional.silu(z)) * mt
    last = h[T if train else T % 2]
    if step:
        return {"y": y[0], "h": last}
    out = {"y": y.transpose(0, 1), "h_T": last.clone()}
    if not train:
        return out
    dread = wide(s["dy"])
    if z is not None:
        sig = torch.sigmoid(z)
        out["dz"] = (dread * read * (sig + z * sig * (1 - sig))).transpose(0, 1)
        dread = dread * torch.nn.functional.silu(z)
    back = torch.zeros_like(h[0]) if s["dh_T"] is None else s["dh_T"].double()
    dA = torch.zeros_like(A)
    dc, db = (torch.empty((T, B, G, N), dtype=torch.float64, device="cuda") for _ in range(2))
    dv, ddelta = torch.empty_like(read), torch.empty_like(read)
    for i in range(T - 1, -1, -1):
        dc[i] = (h[i + 1] * dread[i][..., None]).reshape(B, G, E // G, N).sum(2)
        g = torch.addcmul(back, dread[i][..., None], at(cc, i))
        db[i] = (g * v[i][..., None]).reshape(B, G, E // G, N).sum(2)
        torch.sum(g * at(b, i), -1, out=dv[i])
        back = g.mul_((delta[i][..., None] * A).exp_())
        q = back * h[i]
        torch.sum(q * A, -1, out=ddelta[i])
        dA += (q * delta[i][..., None]).sum(0)
    ddelta += dv * x
    dx = dv * delta
    if s["skip"] is not None:
        dx = dx + s["skip"].double() * dread
        out["dskip"] = (dread * x).sum((0, 1))
    draw_ = (ddelta * torch.sigmoid(raw) if c["softplus"] else ddelta) * mt
    out.update(dx=(dx * mt).transpose(0, 1), ddt=draw_.transpose(0, 1), dA=dA, db=db.transpose(0, 1), dc=dc.transpose(0, 1))
    if s["dt_bias"] is not None:
        out["ddt_bias"] = draw_.sum((0, 1))
    if s["h0"] is not None:
        out["dh0"] = back
    return out


def _exact_norm(s, c):
    train, out = c["op"] == "lnt", {}
    r = s["x"].double()
    if s["residual"] is not None:
        out["r"] = r + s["residual"].double()
        r = out["r"].to(s["residual"].dtype).double()  # the norm is that of the rows as they are kept
    r.requires_grad_(train)
    w, b = (None if s[k] is None else s[k].double().requires_grad_(train) for k in ("w", "b"))
    out["n"] = torch.nn.functional.layer_norm(r, (c["D"],), w, b, EPS)
    if not train:
        return out
    leaf = {"dr": r} if w is None else {"dr": r, "dw": w, "db": b}
    grads = dict(zip(leaf, torch.autograd.grad(out["n"], list(leaf.values()), s["dn"].double())))
    out["n"] = out["n"].detach()
    if s["dr"] is not None:
        grads["dr"] = grads["dr"] + s["dr"].double()
    if c["xdtype"] != c["rdtype"]:
        grads["dx"] = grads["dr"]
    out.update(grads)
    return out
