"""The layer norm, the short convolution and the selective scan as one block uses them: norm with its residual, projection, convolution,
scan with its gate, projection; forward, backward and token by token, captured, on other streams, and what the binding refuses."""
import pytest

import block_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, T, D, E, N, K, RANK = 2, 45, 64, 96, 16, 4, 8


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


@pytest.fixture(scope="module")
def W():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return {"u": n(B, T, D), "r": n(B, T, D), "w": 1 + 0.1 * n(D), "b": 0.1 * n(D), "w_in": n(D, 2 * E) / D ** 0.5, "conv": n(E, K) / 2,
            "conv_b": 0.1 * n(E), "w_x": n(E, RANK + 2 * N) / E ** 0.5, "w_dt": n(RANK, E) / RANK ** 0.5, "dt_bias": n(E) - 3,
            "A": -(torch.arange(1, N + 1, device="cuda").float().expand(E, N)).contiguous(), "skip": 1 + 0.1 * n(E),
            "w_out": n(E, D) / E ** 0.5, "do": n(B, T, D), "dr": n(B, T, D)}


def forward(L, W, u, r, state=None, h0=None, marks=False):
    """The block on whole sequences; everything that its backward pass needs."""
    f = {}
    f["r"], f["n"] = L.layer_norm_fwd(u, W["w"], W["b"], residual=r)
    f["x"], f["z"] = (f["n"] @ W["w_in"]).split(E, -1)  # slices of one projection
    f["y"], f["state"] = L.short_conv_fwd(f["x"], W["conv"], W["conv_b"], state=state)
    f["low"], f["b"], f["c"] = (f["y"] @ W["w_x"]).split([RANK, N, N], -1)
    f["dt"] = f["low"] @ W["w_dt"]
    f["marks"] = L.selective_scan_marks(f["y"], N) if marks else None
    f["s"], f["h"] = L.selective_scan_fwd(f["y"], f["dt"], W["A"], f["b"], f["c"], W["skip"], z=f["z"], dt_bias=W["dt_bias"], h0=h0,
                                          marks=f["marks"])
    f["o"] = f["s"] @ W["w_out"]
    return f


def backward(L, W, f):
    g = L.selective_scan_bwd(f["y"], f["dt"], W["A"], f["b"], f["c"], W["do"] @ W["w_out"].T, f["marks"], W["skip"], z=f["z"],
                             dt_bias=W["dt_bias"])
    dlow = torch.cat([g["ddt"] @ W["w_dt"].T, g["db"], g["dc"]], -1)
    k = L.short_conv_bwd(f["x"], W["conv"], g["dx"] + dlow @ W["w_x"].T, W["conv_b"])
    dn = torch.cat([k["dx"], g["dz"]], -1) @ W["w_in"].T
    e = L.layer_norm_bwd(f["r"], dn, W["w"], W["b"], dr=W["dr"])
    return {"u": e["dx"], "r": e["dr"], "w": e["dw"], "b": e["db"], "conv": k["dw"], "conv_b": k["dbias"], "A": g["dA"], "skip": g["dskip"],
            "dt_bias": g["ddt_bias"]}


def test_block_forward_and_backward(L, W):
    f = forward(L, W, W["u"], W["r"], marks=True)
    got = backward(L, W, f)
    # the same in 64 bits by automatic differentiation
    w = {k: v.double().requires_grad_(k not in ("do", "dr")) for k, v in W.items()}
    r = w["r"] + w["u"]
    n = torch.nn.functional.layer_norm(r, (D,), w["w"], w["b"], 1e-5)
    x, z = (n @ w["w_in"]).split(E, -1)
    pad = torch.nn.functional.pad(x, (0, 0, K - 1, 0))
    y = torch.nn.functional.silu(sum(w["conv"][:, k] * pad[:, k:k + T] for k in range(K)) + w["conv_b"])
    low, b, c = (y @ w["w_x"]).split([RANK, N, N], -1)
    d = torch.nn.functional.softplus(low @ w["w_dt"] + w["dt_bias"])
    h, s = torch.zeros(B, E, N, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        h = torch.exp(d[:, t, :, None] * w["A"]) * h + (d[:, t] * y[:, t])[..., None] * b[:, t, None]
        s.append((h * c[:, t, None]).sum(-1) + w["skip"] * y[:, t])
    o = (torch.stack(s, 1) * torch.nn.functional.silu(z)) @ w["w_out"]
    want = torch.autograd.grad((o * w["do"]).sum() + (r * w["dr"]).sum(), [w[k] for k in got])
    # fp32 through about 200 roundings a path (45 tokens, sums over 64 to 192, norm): 200 * 2^-24 ~ 1.2e-5 of the largest
    near = lambda a, b: (a.double() - b).abs().max() <= 1e-4 * b.abs().max()  # noqa: E731
    assert near(f["o"], o) and near(f["h"], h) and near(f["r"], r)
    for k, v in zip(got, want):
        assert near(got[k], v), k


def test_prompt_then_single_tokens_is_the_sequence(L, W):
    f = forward(L, W, W["u"], W["r"])
    p = forward(L, W, W["u"][:, :20].contiguous(), W["r"][:, :20].contiguous())
    state, h = p["state"], p["h"]
    for t in range(20, T):
        _, n = L.layer_norm_fwd(W["u"][:, t], W["w"], W["b"], residual=W["r"][:, t])
        x, z = (n @ W["w_in"]).split(E, -1)
        y = L.short_conv_step(state, x, W["conv"], W["conv_b"])
        low, b, c = (y @ W["w_x"]).split([RANK, N, N], -1)
        s = L.selective_step(h, y, low @ W["w_dt"], W["A"], b, c, W["skip"], z=z, dt_bias=W["dt_bias"])
        # the products of one row and of all are summed in another order: 64 to 96 terms, 100 * 2^-24 = 6e-6, through two more steps
        assert torch.allclose(s @ W["w_out"], f["o"][:, t], rtol=1e-4, atol=1e-4)
    assert torch.allclose(h, f["h"], rtol=1e-4, atol=1e-4)


def test_captured_and_replayed(L, W):
    """Forms that nothing here has run before, captured at once (16-bit types, other widths, the split time axis), then replayed on
    other values."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").half()  # noqa: E731
    x, dt, b, dy, r = n(1, 800, 40), n(1, 800, 40), n(1, 800, 24), n(1, 800, 40), n(300, 700)
    A, w, taps = -torch.rand(40, 24, device="cuda") - 0.1, torch.ones(700, device="cuda").half(), n(40, 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        marks = L.selective_scan_marks(x, 24)
        y, h = L.selective_scan_fwd(x, dt, A, b, b, marks=marks)
        g = L.selective_scan_bwd(x, dt, A, b, b, dy, marks, dh_T=h)
        k, s = L.short_conv_fwd(x, taps)
        kb = L.short_conv_bwd(x, taps, dy)
        _, m = L.layer_norm_fwd(r, w, w)
        mb = L.layer_norm_bwd(r, m, w, w)
    for seed in (2, 3):
        gen.manual_seed(seed)
        for t in (x, dt, b, dy, r):
            t.copy_(n(*t.shape))
        graph.replay()
        marks2 = L.selective_scan_marks(x, 24)
        y2, h2 = L.selective_scan_fwd(x, dt, A, b, b, marks=marks2)
        g2 = L.selective_scan_bwd(x, dt, A, b, b, dy, marks2, dh_T=h2)
        k2, s2 = L.short_conv_fwd(x, taps)
        kb2 = L.short_conv_bwd(x, taps, dy)
        _, m2 = L.layer_norm_fwd(r, w, w)
        mb2 = L.layer_norm_bwd(r, m2, w, w)
        torch.cuda.synchronize()
        for one, two in ((y, y2), (h, h2), (k, k2), (s, s2), (m, m2), *((g[i], g2[i]) for i in g if g[i] is not None),
                         *((kb[i], kb2[i]) for i in kb if kb[i] is not None), *((mb[i], mb2[i]) for i in mb)):
            assert torch.equal(one, two)


def test_two_streams_at_once_and_given_workspaces(L):
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    sets = [(n(1, 3000, 64), n(1, 3000, 64), n(1, 3000, 16), -torch.rand(64, 16, device="cuda") - 0.1, n(64, 4), n(3000, 5000),
             torch.ones(5000, device="cuda"), *(torch.empty(s, dtype=torch.uint8, device="cuda") for s in
                                                (L.lib().lattice_selective_scan_workspace_bytes(1, 3000, 64, 16, 1, 0),
                                                 L.lib().lattice_selective_scan_workspace_bytes(1, 3000, 64, 16, 1, 1) + 64,
                                                 L.lib().lattice_short_conv_bwd_workspace_bytes(1, 3000, 64, 4),
                                                 L.lib().lattice_layer_norm_bwd_workspace_bytes(3000, 5000)))) for _ in range(2)]

    def work(x, dt, b, A, taps, r, w, w1, w2, w3, w4, stream=None):
        marks = L.selective_scan_marks(x, 16)
        y, h = L.selective_scan_fwd(x, dt, A, b, b, z=x, marks=marks, workspace=w1, stream=stream)
        g = L.selective_scan_bwd(x, dt, A, b, b, y, marks, z=x, dh_T=h, workspace=w2, stream=stream)
        k = L.short_conv_bwd(x, taps, y, workspace=w3, stream=stream)
        m = L.layer_norm_bwd(r, r, w, w, workspace=w4, stream=stream)
        return [y, h, *(v for v in g.values() if v is not None), k["dx"], k["dw"], *m.values()]
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
    for i, s in enumerate(streams):  # the stream named, not entered
        s.wait_stream(torch.cuda.current_stream())
        got[i] = work(*sets[i], stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    L.device_status()


def test_refusals_of_the_binding(L):
    x, dt, A = torch.zeros(2, 8, 32, device="cuda"), torch.zeros(2, 8, 32, device="cuda"), torch.zeros(32, 16, device="cuda")
    b, h, w = torch.zeros(2, 8, 16, device="cuda"), torch.zeros(2, 32, 16, device="cuda"), torch.zeros(32, 4, device="cuda")
    marks, s = L.selective_scan_marks(x, 16), torch.zeros(2, 3, 32, device="cuda")
    bad = [
        (ValueError, lambda: L.selective_scan_fwd(x, dt[:, :7], A, b, b)),
        (ValueError, lambda: L.selective_scan_fwd(x, dt, A, b, b[:, :, :8])),
        (ValueError, lambda: L.selective_scan_fwd(x, dt, A[:31], b, b)),
        (ValueError, lambda: L.selective_scan_fwd(x, dt, A, b.unflatten(-1, (2, 8)), b.unflatten(-1, (2, 8)))),
        (ValueError, lambda: L.selective_scan_fwd(x, dt, A, b[:, :, None].expand(2, 8, 3, 16), b[:, :, None].expand(2, 8, 3, 16))),
        (ValueError, lambda: L.selective_scan_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), dt, A, b, b)),
        (ValueError, lambda: L.selective_scan_fwd(x, dt, A.T.contiguous().T, b, b)),
        (ValueError, lambda: L.selective_scan_bwd(x, dt, A, b, b, x, marks[:, :0])),
        (ValueError, lambda: L.selective_step(h[:1], x[:, 0], dt[:, 0], A, b[:, 0], b[:, 0])),
        (ValueError, lambda: L.short_conv_fwd(x, w[:31])),
        (ValueError, lambda: L.short_conv_fwd(x, w, act="gelu")),
        (ValueError, lambda: L.short_conv_fwd(x, w, state=s[:, :2])),
        (ValueError, lambda: L.short_conv_step(s[:, :2], x[:, 0], w)),
        (ValueError, lambda: L.layer_norm_fwd(x, torch.ones(31, device="cuda"))),
        (ValueError, lambda: L.layer_norm_fwd(x, r_out=x)),
        (TypeError, lambda: L.selective_scan_fwd(x, dt.bfloat16(), A, b, b)),
        (TypeError, lambda: L.selective_scan_fwd(x, dt, A, b.bfloat16(), b)),
        (TypeError, lambda: L.selective_scan_fwd(x, dt, A.bfloat16(), b, b)),
        (TypeError, lambda: L.selective_scan_fwd(x.double(), dt, A, b, b)),
        (TypeError, lambda: L.selective_scan_fwd(x, dt, A, b, b, lengths=torch.zeros(2, device="cuda", dtype=torch.int64))),
        (TypeError, lambda: L.selective_scan_fwd(x, dt, A, b, b, workspace=3)),
        (TypeError, lambda: L.short_conv_fwd(x, w, torch.zeros(32, device="cuda").bfloat16())),
        (TypeError, lambda: L.short_conv_fwd(x, w, state=s.bfloat16())),
        (TypeError, lambda: L.layer_norm_fwd(x, torch.ones(32, device="cuda").bfloat16())),
        (TypeError, lambda: L.layer_norm_bwd(x.bfloat16(), x.bfloat16(), x_dtype=torch.float16)),
    ]
    for error, f in bad:
        with pytest.raises(error):
            f()
    codes = [
        (L.ERR_INVALID_ARG, lambda: L.selective_scan_fwd(x, dt, A, b, b, y=x)),
        (L.ERR_INVALID_ARG, lambda: L.selective_step(h, x[:, 0], dt[:, 0], A, b[:, 0], b[:, 0], y=h.view(-1)[:64].view(2, 32))),
        (L.ERR_INVALID_ARG, lambda: L.short_conv_fwd(x, w, y=x)),
        (L.ERR_INVALID_ARG, lambda: L.layer_norm_fwd(x, n_out=x)),
        (L.ERR_INVALID_ARG, lambda: L.layer_norm_fwd(x, eps=0.0)),
        (L.ERR_INVALID_ARG, lambda: L.short_conv_bwd(x, w, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (L.ERR_UNSUPPORTED, lambda: L.short_conv_fwd(x, torch.zeros(32, 9, device="cuda"))),
        (L.ERR_UNSUPPORTED, lambda: L.selective_scan_fwd(x, dt, torch.zeros(32, 129, device="cuda"), torch.zeros(2, 8, 129, device="cuda"),
                                                         torch.zeros(2, 8, 129, device="cuda"))),
        (L.ERR_UNSUPPORTED, lambda: L.layer_norm_fwd(torch.zeros(1, 16385, device="cuda"))),
    ]
    for code, f in codes:
        with pytest.raises(L.LatticeError) as e:
            f()
        assert e.value.code == code


def test_sizes_past_a_c_int_are_refused(L):
    """They would reach the library as their lower 32 bits: 3 tokens, 1 state."""
    x = torch.zeros(1, 1, 1, device="cuda").bfloat16()
    many, A, b = x.expand(1, (1 << 32) + 3, 1), torch.zeros(1, 1, device="cuda"), x.expand(1, (1 << 32) + 3, 1)
    wide = torch.empty(1, (1 << 32) + 64, dtype=torch.bfloat16, device="cuda")
    for f in (lambda: L.selective_scan_fwd(many, many, A, b, b), lambda: L.short_conv_fwd(many, A.bfloat16()), lambda: L.layer_norm_fwd(wide),
              lambda: L.short_conv_fwd(x, wide)):
        with pytest.raises(L.LatticeError) as e:
            f()
        assert e.value.code == L.ERR_UNSUPPORTED


def test_what_stands_around_the_outputs_is_left_alone(L):
    """Outputs inside larger buffers, at odd widths: nothing before or behind them changes."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    for C in (33, 40):
        x, b, A = n(2, 50, C), n(2, 50, 7), -torch.rand(C, 7, device="cuda")

        def framed(shape, dtype):
            size = 1
            for k in shape:
                size *= k
            whole = torch.full((size + 128,), 7.0, dtype=dtype, device="cuda")
            return whole, whole[64:64 + size].view(shape)
        wy, y = framed((2, 50, C), torch.bfloat16)
        wh, h = framed((2, C, 7), torch.float32)
        wm, marks = framed((2, 7, C, 7), torch.float32)
        L.selective_scan_fwd(x, x, A, b, b, y=y, h_out=h, marks=marks)
        wk, k = framed((2, 50, C), torch.bfloat16)
        ws, s = framed((2, 3, C), torch.bfloat16)
        L.short_conv_fwd(x, n(C, 4), y=k, state_out=s)
        wn, norm = framed((2, 50, C), torch.bfloat16)
        L.layer_norm_fwd(x, n_out=norm)
        for whole in (wy, wh, wm, wk, ws, wn):
            assert bool((whole[:64] == 7).all()) and bool((whole[-64:] == 7).all())


def test_the_documented_calls(L):
    """The calls on the front page, as they stand there."""
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        example, = re.findall(r"```py\n(.*?)```", f.read(), re.S)
    gen = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    b, t, d, e, k = 3, 130, 64, 128, 16
    names = {"lattice": L, "u": n(b, t, d).bfloat16(), "r": n(b, t, d), "w_norm": n(d), "b_norm": n(d), "x": n(b, t, e).bfloat16(),
             "z": n(b, t, e).bfloat16(), "w_conv": n(e, 4), "b_conv": n(e), "dt": n(b, t, e).bfloat16(), "A": -n(e, k).abs(),
             "b": n(b, t, k).bfloat16(), "c": n(b, t, k).bfloat16(), "skip": n(e), "dt_bias": n(e) - 3, "dy": n(b, t, e).bfloat16(),
             "dn": n(b, t, d).bfloat16(), "dr": n(b, t, d), "x_t": n(b, e).bfloat16(), "z_t": n(b, e).bfloat16(), "dt_t": n(b, e).bfloat16(),
             "b_t": n(b, k).bfloat16(), "c_t": n(b, k).bfloat16()}
    exec(example, names)
    assert set(names["g_scan"]) == {"dx", "ddt", "dA", "db", "dc", "dskip", "dz", "ddt_bias", "dh0"}
    assert names["y_t"].shape == (b, e) and bool(torch.isfinite(names["y_t"].float()).all())
    L.device_status()
