"""The norms after and before a block on the GPU against their 64-bit forms."""
import pytest

import norm_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


def make(shape, dtype="bf16", ydtype=None, rdtype=None, wdtype="f32", gate=True, residual=True, post_w=True, pre_w=True, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    D = shape[-1]
    return {"y": (0.7 * n(*shape)).to(DT[ydtype or dtype]), "gate": n(*shape).mul(1.5).to(DT[dtype]) if gate else None,
            "residual": (2 * n(*shape)).to(DT[rdtype or dtype]) if residual else None,
            "w_post": (1 + 0.2 * n(D)).to(DT[wdtype]) if post_w else None,
            "w_pre": (1 + 0.2 * n(D)).to(DT[wdtype]) if pre_w else None,
            "dr": n(*shape).to(DT[rdtype or dtype] if residual else DT[dtype]), "dn": n(*shape).to(DT[dtype]), "dtype": DT[dtype]}


def both(L, t, act="gelu", pre=True, post=True, scale=0.5, eps=1e-6, dr=True):
    kw = dict(gate=t["gate"], act=act, residual=t["residual"], scale=scale, eps=eps)
    r, n = L.block_norm_fwd(t["y"], t["w_post"], w_pre=t["w_pre"] if pre else None, pre_norm=pre, post_norm=post,
                            out_dtype=t["dtype"], **kw)
    ref, _ = R.forward(t["y"], t["w_post"], t["gate"], act, t["residual"], t["w_pre"] if pre else None, pre, post, scale, eps)
    R.check(r, ref, "r")
    assert r.dtype == (t["dtype"] if t["residual"] is None else t["residual"].dtype)
    got = {"r": r}
    if pre:
        R.check(n, ref, "n")
        assert n.dtype == t["dtype"]
        got["n"] = n
    else:
        assert n is None
    g = L.block_norm_bwd(t["y"], t["w_post"], dr=t["dr"] if dr else None, dn=t["dn"] if pre else None,
                         w_pre=t["w_pre"] if pre else None, post_norm=post, **kw)
    ref = R.backward(t["y"], t["w_post"], t["gate"], act, t["residual"], t["w_pre"] if pre else None, post, scale, eps,
                     t["dr"] if dr else None, t["dn"] if pre else None)
    for k, have in (("dy", True), ("dgate", t["gate"] is not None), ("dresidual", t["residual"] is not None),
                    ("dw_post", t["w_post"] is not None), ("dw_pre", pre and t["w_pre"] is not None)):
        if have:
            R.check(g[k], ref, k)
            got[k] = g[k]
        else:
            assert g[k] is None
    return got


WIDTHS = [1, 2, 7, 8, 9, 24, 63, 64, 100, 128, 255, 256, 257, 511, 520, 1000, 1024, 1528, 2047, 2048, 2056, 4096, 4097, 8192,
          8200, 16383, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,ydtype,rdtype", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f16", "f32", "f32")])
def test_widths_and_types(L, D, dtype, ydtype, rdtype):
    both(L, make((5, D), dtype, ydtype, rdtype, wdtype="f32" if D % 2 else dtype, seed=D))


@pytest.mark.parametrize("N", [1, 2, 3, 31, 33, 257, 5000])
@pytest.mark.parametrize("D", [16, 64, 72, 128, 640])
def test_row_counts(L, N, D):
    both(L, make((N, D), "bf16", "f32", "f32", seed=N + D))


@pytest.mark.parametrize("act", ["gelu", "silu", "sigmoid"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_forms(L, act, post, pre, residual):
    for gate in (True, False):
        for D in (96, 1096):
            both(L, make((9, D), "bf16", "f32", gate=gate, residual=residual, seed=3), act, pre, post, scale=-1.25)
            both(L, make((9, D), "f32", gate=gate, residual=residual, seed=4), act, pre, post)


def test_without_weights_and_cotangents(L):
    for D in (40, 2888):
        both(L, make((6, D), post_w=False, pre_w=False, seed=5))
        both(L, make((6, D), post_w=False, seed=6), dr=False)
        both(L, make((6, D), pre_w=False, seed=7), pre=False)


def test_no_rows(L):
    t = make((0, 64))
    r, n = L.block_norm_fwd(t["y"], t["w_post"], gate=t["gate"], residual=t["residual"], w_pre=t["w_pre"])
    assert r.shape == (0, 64) and n.shape == (0, 64)
    g = L.block_norm_bwd(t["y"], t["w_post"], dr=t["dr"], dn=t["dn"], gate=t["gate"], residual=t["residual"], w_pre=t["w_pre"])
    assert (g["dw_post"] == 0).all() and (g["dw_pre"] == 0).all() and g["dy"].shape == (0, 64)


def test_rows_of_nothing(L):
    """All-zero rows: the norms' epsilon keeps them finite."""
    t = make((4, 128), "f32", seed=8)
    t["y"][1], t["residual"][1] = 0, 0
    t["y"][2] = 0
    both(L, t)


@pytest.mark.parametrize("N,D", [(5, 64), (7, 63), (3, 200), (3, 2048), (2, 9000)])
def test_rows_of_nothing_with_a_tiny_epsilon(L, N, D):
    """1/sqrt(eps) to the third power is past fp32's range here, for zero rows, and in the threads
    of a CTA that have no row, too."""
    for post in (True, False):
        t = make((N, D), "f32", seed=D)
        both(L, t, post=post, eps=1e-30)
        t["y"][1], t["residual"][1] = 0, 0
        both(L, t, post=post, eps=1e-30)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(5, 64), (3, 2048), (4, 1001), (2, 9000)])
@pytest.mark.parametrize("size", [1e13, 1e15, 1e17])
def test_rows_of_large_values(L, N, D, dtype, size):
    """Their inverse root mean square to the third power is below fp32's range; their gradients are not.
    A row's sum of squares has to be within it, too: 9000 values of deviation 2e17 have 3.6e38, past
    the 3.4e38 that fp32 holds, and are not supported."""
    if D * (2 * size) ** 2 > 3.4e38:
        pytest.skip("the sum of squares is past fp32's range")
    for post, residual in ((True, True), (False, True), (True, False)):
        t = make((N, D), dtype, seed=D, residual=residual)
        t["y"] *= size
        if residual:
            t["residual"] *= size
            t["dr"] /= size
        both(L, t, post=post)
        both(L, t, post=post, pre=False)


def test_groups_of_wider_rows(L):
    B, T, H, d = 2, 6, 3, 32
    t = make((B, T, H, d), "bf16", seed=9)
    want = both(L, t)
    wide = torch.zeros((B, T, 2, H, d), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1] = t["gate"]
    t["gate"] = wide[:, :, 1]
    got = both(L, t)
    assert all(torch.equal(got[k], want[k]) for k in want)
    t = make((10, 48), "bf16", seed=10)
    want = both(L, t)
    for k in ("y", "gate", "residual", "dr", "dn"):
        w = torch.zeros((10, 48 + 7), dtype=t[k].dtype, device="cuda")
        w[:, 3:51] = t[k]
        t[k] = w[:, 3:51]
    got = both(L, t)
    for k in want:  # other reads, and other sums of a row
        assert torch.allclose(got[k].float(), want[k].float(), rtol=1e-2, atol=1e-2)
    t = make((4, 5, 24), "f32", seed=11)
    t["residual"] = t["residual"][:, :1].expand(4, 5, 24)  # no stride that groups of rows have
    with pytest.raises(ValueError):
        both(L, t)


@pytest.mark.parametrize("N,D", [(9, 1), (3000, 3), (5000, 12), (4, 50), (2600, 129), (700, 250), (5, 255), (1500, 257),
                                 (600, 2055), (301, 4090), (450, 4095), (200, 4097), (90, 8187), (75, 16377), (75, 16378)])
@pytest.mark.parametrize("dtype,ydtype,rdtype", [("bf16", "bf16", "f32"), ("f32", "f32", "f32"), ("f16", "f32", "f16")])
def test_widths_that_are_no_multiple_of_a_vector(L, N, D, dtype, ydtype, rdtype):
    both(L, make((N, D), dtype, ydtype, rdtype, seed=N + D))
    both(L, make((N, D), dtype, ydtype, rdtype, gate=False, residual=False, seed=N + D + 1), pre=False)


@pytest.mark.parametrize("more", [8, 16, 4, 3])
def test_groups_of_odd_rows(L, more):
    """Rows that start where those of whole arrays would (8, 16; 4 in fp32), and elsewhere."""
    G, D, groups = 5, 77, 130
    t = make((groups, G, D), "bf16", "f32", "f32", seed=21)
    want = both(L, t)
    for k in ("y", "gate", "residual", "dr", "dn"):
        w = torch.full((groups, G * D + more), float("nan"), dtype=t[k].dtype, device="cuda")
        w[:, :G * D] = t[k].flatten(1)
        t[k] = w[:, :G * D].view(groups, G, D)
    got = both(L, t)
    if more % 8 == 0:
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("D", [5, 300, 999, 5000, 9001])
def test_rows_that_start_anywhere(L, D):
    N = 23
    t = make((N, D), "bf16", "f32", "f32", seed=D)
    for k in ("y", "gate", "residual", "dr", "dn"):
        w = torch.full((N * D + 1,), float("nan"), dtype=t[k].dtype, device="cuda")
        w[1:] = t[k].flatten()
        t[k] = w[1:].view(N, D)
    both(L, t)


def test_odd_rows_keep_to_themselves(L):
    """What stands around a row is neither read into it nor written."""
    for N, D in ((40, 37), (700, 259), (20, 5003)):
        t = make((N, D), "bf16", "f32", "f32", seed=22)
        kw = dict(act="gelu", scale=0.5)
        want, n = L.block_norm_fwd(t["y"], t["w_post"], gate=t["gate"], residual=t["residual"], w_pre=t["w_pre"], **kw)
        for i in (0, N // 2, N - 1):
            bad = {k: t[k].clone() for k in ("y", "gate", "residual", "dr", "dn")}
            for k in bad:
                bad[k][i] = float("nan")
            r, m = L.block_norm_fwd(bad["y"], t["w_post"], gate=bad["gate"], residual=bad["residual"], w_pre=t["w_pre"], **kw)
            keep = [j for j in range(N) if j != i]
            assert torch.equal(r[keep], want[keep]) and torch.equal(m[keep], n[keep])
            one = L.block_norm_bwd(t["y"], t["w_post"], gate=t["gate"], residual=t["residual"], w_pre=t["w_pre"], dr=t["dr"],
                                   dn=t["dn"], **kw)
            two = L.block_norm_bwd(bad["y"], t["w_post"], gate=bad["gate"], residual=bad["residual"], w_pre=t["w_pre"],
                                   dr=bad["dr"], dn=bad["dn"], **kw)
            for k in ("dy", "dgate", "dresidual"):
                assert torch.equal(two[k][keep], one[k][keep]) and two[k][i].isnan().any()
        room = torch.full((N * D + 32,), 7.0, device="cuda")
        out = room[16:16 + N * D].view(N, D)
        out.copy_(t["residual"])
        r, m = L.block_norm_fwd(t["y"], t["w_post"], gate=t["gate"], residual=out, w_pre=t["w_pre"], r_out=out, **kw)
        assert torch.equal(r, want) and torch.equal(m, n)
        assert (room[:16] == 7).all() and (room[16 + N * D:] == 7).all()


def test_residual_in_place(L):
    t = make((7, 256), "bf16", rdtype="f32", seed=12)
    want, n = L.block_norm_fwd(t["y"], t["w_post"], residual=t["residual"], w_pre=t["w_pre"])
    r, m = L.block_norm_fwd(t["y"], t["w_post"], residual=t["residual"], w_pre=t["w_pre"], r_out=t["residual"])
    assert r is t["residual"] and torch.equal(r, want) and torch.equal(m, n)


def test_not_a_number_stays_in_its_row(L):
    for D in (64, 2048):
        t = make((5, D), "bf16", seed=13)
        t["y"][2, 3] = float("nan")
        r, n = L.block_norm_fwd(t["y"], t["w_post"], residual=t["residual"], w_pre=t["w_pre"])
        bad = torch.isnan(n.float()).any(-1)
        assert bad.tolist() == [False, False, True, False, False]


def test_the_same_call_gives_the_same_bits(L):
    for shape in ((3000, 64), (700, 2048)):
        t = make(shape, "bf16", seed=14)
        one, two = both(L, t), both(L, t)
        assert all(torch.equal(one[k], two[k]) for k in one)


@pytest.mark.parametrize("N,D", [(1, 1), (300, 64), (3000, 100), (90, 2056), (40, 8187), (75, 16384)])
def test_a_callers_workspace(L, N, D):
    """Of the stated size, whatever it holds: the same bits as with the library's own. Nothing
    behind it is written, and a smaller one is refused."""
    t = make((N, D), "bf16", "f32", "f32", seed=N)
    kw = dict(gate=t["gate"], residual=t["residual"], w_pre=t["w_pre"], dr=t["dr"], dn=t["dn"])
    want = L.block_norm_bwd(t["y"], t["w_post"], **kw)
    need = L.lib().lattice_block_norm_bwd_workspace_bytes(N, D)
    room = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    room[need // 4:] = 7.0
    for _ in range(2):
        got = L.block_norm_bwd(t["y"], t["w_post"], workspace=room[:need // 4], **kw)
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert (room[need // 4:] == 7).all()
    with pytest.raises(L.LatticeError) as e:
        L.block_norm_bwd(t["y"], t["w_post"], workspace=room[:need // 4 - 1], **kw)
    assert e.value.code == L.ERR_INVALID_ARG
    with pytest.raises(L.LatticeError):  # over an input
        L.block_norm_bwd(t["y"], t["w_post"], workspace=t["residual"] if t["residual"].numel() * 4 >= need else t["w_post"], **kw)
    small = L.block_norm_bwd(t["y"], gate=t["gate"], residual=t["residual"], dr=t["dr"])  # no weights: none is needed
    assert small["dw_post"] is None and small["dw_pre"] is None


def test_streams_and_graphs(L):
    t = make((300, 1024), "bf16", seed=15)
    kw = dict(gate=t["gate"], residual=t["residual"], w_pre=t["w_pre"])
    want = L.block_norm_bwd(t["y"], t["w_post"], dr=t["dr"], dn=t["dn"], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = L.block_norm_bwd(t["y"], t["w_post"], dr=t["dr"], dn=t["dn"], stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, n = L.block_norm_fwd(t["y"], t["w_post"], **kw)
        got = L.block_norm_bwd(t["y"], t["w_post"], dr=t["dr"], dn=t["dn"], **kw)
    other = make((300, 1024), "bf16", seed=16)
    for k in ("y", "gate", "residual", "dr", "dn"):
        t[k].copy_(other[k])
    graph.replay()
    want = L.block_norm_bwd(t["y"], t["w_post"], dr=t["dr"], dn=t["dn"], **kw)
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert torch.equal(r, L.block_norm_fwd(t["y"], t["w_post"], **kw)[0])


def test_a_large_batch_of_rows(L):
    """More rows than CTAs at once, with offsets past 2^31 bytes."""
    t = make((70000, 8192), "bf16", gate=False, seed=17)
    r, n = L.block_norm_fwd(t["y"], t["w_post"], residual=t["residual"], w_pre=t["w_pre"])
    pick = slice(69990, 70000)
    ref, _ = R.forward(t["y"][pick], t["w_post"], None, "gelu", t["residual"][pick], t["w_pre"], True, True, 1.0, 1e-6)
    R.check(r[pick], ref, "r")
    R.check(n[pick], ref, "n")
