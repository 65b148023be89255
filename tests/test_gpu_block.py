"""The state recurrences and the norms as one layer uses them: norm before, projections, the
Lattice scan beside the gated recurrence, norm and gate on the read-out, output projection,
scaled residual and the next norm; forward, backward and token by token."""
import pytest

import gated_ref
import norm_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, T, H, d, m = 2, 70, 2, 64, 64
D = H * d


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


@pytest.fixture(scope="module")
def W():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return {"r": n(B, T, D), "w_in": 1 + 0.1 * n(D), "proj": n(D, 3 * D) / D ** 0.5, "w_post": 1 + 0.1 * n(d),
            "out": n(D, D) / D ** 0.5, "w_res": 1 + 0.1 * n(D), "w_next": 1 + 0.1 * n(D), "dr": n(B, T, D), "dn": n(B, T, D),
            "c": torch.sigmoid(n(B, T, H, m)), "q": n(B, T, H, m) / m ** 0.5, "mu": torch.sigmoid(3 + n(B, T, H)),
            "S0": torch.nn.functional.normalize(n(B, H, m, d), dim=-1)}


def split(p):
    return [v.unflatten(-1, (H, d)) for v in p.split(D, -1)]  # x, z, gate: slices of one projection


def test_layer_forward_and_backward(L, W):
    n0, _ = L.block_norm_fwd(W["r"], W["w_in"])
    x, z, g = split(n0 @ W["proj"])
    marks = L.gated_scan_marks(x)
    y, _ = L.gated_scan_fwd(x, z, write="unit", marks=marks)
    o, none = L.block_norm_fwd(y, W["w_post"], gate=g)
    assert none is None
    u = o.flatten(-2) @ W["out"]
    r1, n1 = L.block_norm_fwd(u, W["w_res"], residual=W["r"], w_pre=W["w_next"], scale=0.5)
    # backward, piece by piece
    a = L.block_norm_bwd(u, W["w_res"], residual=W["r"], w_pre=W["w_next"], scale=0.5, dr=W["dr"], dn=W["dn"])
    do = (a["dy"] @ W["out"].T).unflatten(-1, (H, d))
    b = L.block_norm_bwd(y, W["w_post"], gate=g, dr=do)
    c = L.gated_scan_bwd(x, z, b["dy"], marks, write="unit")
    dn0 = torch.cat([v.flatten(-2) for v in (c["dx"], c["dz"], b["dgate"])], -1) @ W["proj"].T
    e = L.block_norm_bwd(W["r"], W["w_in"], dr=dn0)
    dr = a["dresidual"] + e["dy"]

    # the same in 64 bits by automatic differentiation
    leaf = {k: W[k].double().requires_grad_() for k in ("r", "w_in", "proj", "w_post", "out", "w_res", "w_next")}
    norm = lambda t, w: t / (t.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    x8, z8, g8 = split(norm(leaf["r"], leaf["w_in"]) @ leaf["proj"])
    gate = torch.sigmoid(z8)
    s = torch.sqrt(torch.sigmoid(-z8) * (1 + gate))
    h, ys = torch.zeros(B, H, d, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        h = gate[:, t] * h + s[:, t] * x8[:, t]
        ys.append(h)
    o8 = norm(torch.stack(ys, 1), leaf["w_post"]) * torch.nn.functional.gelu(g8)
    r8 = leaf["r"] + 0.5 * norm(o8.flatten(-2) @ leaf["out"], leaf["w_res"])
    n8 = norm(r8, leaf["w_next"])
    grads = dict(zip(leaf, torch.autograd.grad((r8 * W["dr"]).sum() + (n8 * W["dn"]).sum(), list(leaf.values()))))
    # fp32 through about 150 roundings a path (70 tokens, two sums over 128, norms): 150 * 2^-24 ~ 1e-5 of the largest
    near = lambda a, b: (a.double() - b).abs().max() <= 1e-4 * b.abs().max()  # noqa: E731
    assert near(r1, r8) and near(n1, n8)
    assert near(dr, grads["r"]) and near(a["dw_pre"], grads["w_next"]) and near(a["dw_post"], grads["w_res"])
    assert near(b["dw_post"], grads["w_post"]) and near(e["dw_post"], grads["w_in"])


def test_token_by_token_is_the_sequence(L, W):
    """The decode forms of both recurrences and the norms on one row per sequence. fp32 over 70
    tokens: each commits a few 2^-24 of the state, 70 * 16 * 2^-24 = 7e-5; the Lattice state
    turns with its errors too, and its scan tests allow ten times that."""
    n0, _ = L.block_norm_fwd(W["r"], W["w_in"])
    x, z, g = split(n0 @ W["proj"])
    y, _ = L.gated_scan_fwd(x, z)
    o, _ = L.block_norm_fwd(y, W["w_post"], gate=g)
    yl, _ = L.scan_fwd(x.contiguous(), W["c"], W["q"], W["mu"], W["S0"])
    ol, _ = L.block_norm_fwd(yl, W["w_post"], gate=g)
    h, S = torch.zeros(B, H, d, device="cuda"), W["S0"].clone()
    for t in range(T):
        yt = L.gated_step(h, x[:, t], z[:, t])
        ot, _ = L.block_norm_fwd(yt, W["w_post"], gate=g[:, t])
        assert torch.allclose(ot, o[:, t], rtol=1e-4, atol=1e-4)
        yt = L.step(S, *(v[:, t].contiguous() for v in (x, W["c"], W["q"], W["mu"])))
        ot, _ = L.block_norm_fwd(yt, W["w_post"], gate=g[:, t])
        assert torch.allclose(ot, ol[:, t], rtol=1e-3, atol=1e-3)


def test_first_use_inside_a_capture(L):
    """A form of each operator that nothing in this file has run before, captured at once."""
    x = torch.randn(3, 700, 1, 96, device="cuda").half()
    z = torch.randn(3, 700, 1, 96, device="cuda")
    r = torch.randn(3, 9000, device="cuda").half()
    w = torch.ones(9000, device="cuda").half()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        marks = L.gated_scan_marks(x)
        y, h = L.gated_scan_fwd(x, z, gate="logit", write="unit", tau=0.7, marks=marks)
        g = L.gated_scan_bwd(x, z, y, marks, dh_T=h, gate="logit", write="unit", tau=0.7)
        a, n = L.block_norm_fwd(r, w, gate=r, act="sigmoid", residual=r, w_pre=w)
        b = L.block_norm_bwd(r, w, gate=r, act="sigmoid", residual=r, w_pre=w, dr=a, dn=n)
    graph.replay()
    torch.cuda.synchronize()
    ref = gated_ref.scan(x, z, None, "logit", "unit", 0.7, None, y, h)
    for k, v in (("y", y), ("h_T", h), ("dx", g["dx"]), ("dz", g["dz"]), ("dh0", g["dh0"])):
        gated_ref.check(v, ref, k)
    ref, _ = norm_ref.forward(r, w, r, "sigmoid", r, w, True, True, 1.0, 1e-6)
    norm_ref.check(a, ref, "r")
    norm_ref.check(n, ref, "n")
    ref = norm_ref.backward(r, w, r, "sigmoid", r, w, True, 1.0, 1e-6, a, n)
    for k, v in b.items():
        norm_ref.check(v, ref, k)


def test_two_streams_at_once(L):
    """The same calls on two streams give what they give alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    sets = [(n(2, 3000, 2, 64), n(2, 3000, 2, 64), n(4000, 5000), torch.ones(5000, device="cuda")) for _ in range(2)]

    def work(x, z, r, w):
        marks = L.gated_scan_marks(x)
        y, h = L.gated_scan_fwd(x, z, marks=marks)
        g = L.gated_scan_bwd(x, z, y, marks, dh_T=h)
        k = L.block_norm_bwd(r, w, residual=r, w_pre=w, dr=r, dn=r)
        return [y, h, g["dx"], g["dz"], g["dh0"], k["dy"], k["dw_post"], k["dw_pre"]]
    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = work(*sets[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    L.device_status()


def test_refusals_of_the_binding(L):
    x = torch.zeros(2, 8, 2, 32, device="cuda")
    h = torch.zeros(2, 2, 32, device="cuda")
    with pytest.raises(ValueError):
        L.gated_scan_fwd(x, x[:, :7])
    with pytest.raises(TypeError):
        L.gated_scan_fwd(x, x.bfloat16())
    with pytest.raises(TypeError):
        L.gated_scan_fwd(x.double(), x.double())
    with pytest.raises(ValueError):
        L.gated_scan_fwd(x.transpose(2, 3).contiguous().transpose(2, 3), x)
    with pytest.raises(ValueError):
        L.gated_scan_fwd(x, x, gate="sigmoid")
    with pytest.raises(L.LatticeError) as e:
        L.gated_scan_fwd(x, x, tau=0.0)
    assert e.value.code == L.ERR_INVALID_ARG
    with pytest.raises(L.LatticeError) as e:
        L.gated_scan_fwd(x.flatten(2).unsqueeze(2)[..., :48].contiguous(), x[:, :, :1, 0])
    assert e.value.code == L.ERR_UNSUPPORTED  # a gate per head of 48
    with pytest.raises(TypeError):
        L.gated_scan_fwd(x, x, lengths=torch.zeros(2, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        L.gated_step(h, x[:, 0], x[:, 0], h_out=h[:1])
    with pytest.raises(L.LatticeError):
        L.gated_step(h, x[:, 0], x[:, 0], y=h)  # the output over the state
    r = torch.zeros(4, 64, device="cuda")
    with pytest.raises(TypeError):
        L.block_norm_fwd(r, torch.ones(64, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        L.block_norm_fwd(r, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        L.block_norm_fwd(r, act="relu", gate=r)
    with pytest.raises(L.LatticeError):
        L.block_norm_fwd(r, eps=0.0)
    with pytest.raises(ValueError):
        L.block_norm_bwd(r, w_pre=torch.ones(64, device="cuda"), dr=r)
    with pytest.raises(L.LatticeError):
        L.block_norm_fwd(torch.zeros(1, 16385, device="cuda"))


def test_sizes_past_a_c_int_are_refused(L):
    """They would reach the library as their lower 32 bits: 3 tokens, 64 columns."""
    x = torch.zeros(1, 1, 1, 1, device="cuda").bfloat16()
    many = x.expand(1, (1 << 32) + 3, 1, 1)
    with pytest.raises(L.LatticeError) as e:
        L.gated_scan_fwd(many, many)
    assert e.value.code == L.ERR_UNSUPPORTED
    with pytest.raises(L.LatticeError) as e:
        L.gated_scan_bwd(many, many, many, torch.zeros(1, 1, 1, 1, device="cuda"))
    assert e.value.code == L.ERR_UNSUPPORTED
    wide = torch.empty(1, (1 << 32) + 64, dtype=torch.bfloat16, device="cuda")
    for f in (lambda: L.block_norm_fwd(wide), lambda: L.block_norm_bwd(wide, dr=wide)):
        with pytest.raises(L.LatticeError) as e:
            f()
        assert e.value.code == L.ERR_UNSUPPORTED


def test_the_documented_calls(L):
    """The example of the project's front page, as it stands there, on a batch of three: its calls run,
    and the token that it decodes goes on from the sequence's state."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        example, = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    b, t, heads, width, slots = 3, 130, 2, 64, 64
    names = {"x": n(b, t, heads, width).bfloat16(), "c": torch.sigmoid(n(b, t, heads, slots)),
             "q": n(b, t, heads, slots).bfloat16(), "mu": torch.sigmoid(n(b, t, heads)),
             "S0": torch.nn.functional.normalize(n(b, heads, slots, width), dim=-1), "dS_T": n(b, heads, slots, width),
             "x_t": n(b, heads, width).bfloat16(), "c_t": torch.sigmoid(n(b, heads, slots)),
             "q_t": n(b, heads, slots).bfloat16(), "mu_t": torch.sigmoid(n(b, heads)),
             "z": (n(b, t, heads, width) + 2).bfloat16(), "h0": n(b, heads, width), "dh": n(b, heads, width),
             "z_t": (n(b, heads, width) + 2).bfloat16(), "w_head": n(width), "gate": n(b, t, heads, width).bfloat16(),
             "p": n(b, t, heads * width).bfloat16(), "w_post": n(heads * width), "w_pre": n(heads * width),
             "r0": n(b, t, heads * width), "dr": n(b, t, heads * width), "dn": n(b, t, heads * width).bfloat16()}
    names["dy"] = n(b, t, heads, width)
    for line in example.splitlines():
        if line.startswith("g = lattice.gated_scan_bwd"):  # here dy has x's type
            names["dy"] = names["dy"].bfloat16()
        exec(line, names)
    both = torch.cat([names["x"], names["x_t"].unsqueeze(1)], 1), torch.cat([names["z"], names["z_t"].unsqueeze(1)], 1)
    ref = gated_ref.scan(*both, names["h0"], "logit", "unit", 0.125)
    gated_ref.check(names["h"], ref, "h_T")
    gated_ref.check(names["y_t"].unsqueeze(1), {"y": ref["y"][:, -1:], "b_y": ref["b_y"][:, -1:]}, "y")
    assert set(names["g"]) == {"dy", "dgate", "dresidual", "dw_post", "dw_pre"}
    L.device_status()
