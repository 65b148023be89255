"""The layer norm on the GPU against the 64-bit form, at the widths where vectors, warps, CTAs and clusters end.

Units of 2^-24 of the terms' magnitude: a row's sums are taken in trees of at most 8 + 5 + 5 + 2 additions, twice (the mean, the
variance), the reciprocal root and the products add 8: 64 covers both directions. The weights' gradients add the rows of a CTA one by
one, then the CTAs."""
import pytest

import block_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


def make(N, D, dtype="f32", xdtype=None, rdtype=None, wdtype=None, residual=True, affine=True, mean=0.5, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    xt = DT[xdtype or dtype]
    rt = DT[rdtype or dtype] if residual else xt
    return {"x": (n(N, D) + mean).to(xt), "residual": (n(N, D) * 2).to(rt) if residual else None,
            "w": (1 + 0.3 * n(D)).to(DT[wdtype or dtype]) if affine else None, "b": n(D).to(DT[wdtype or dtype]) if affine else None,
            "dn": n(N, D).to(DT[dtype]), "dr": n(N, D).to(rt), "dtype": DT[dtype]}


def check(L, t, dr=True, eps=1e-5):
    r, n = L.layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["residual"], eps=eps, out_dtype=t["dtype"])
    g_r = t["dr"] if dr else None
    got = L.layer_norm_bwd(r, t["dn"], t["w"], t["b"], dr=g_r, eps=eps, x_dtype=t["x"].dtype)
    want, mag = R.layer(t["x"], t["w"], t["b"], t["residual"], eps, t["dn"], g_r)
    if t["residual"] is None:
        assert r is t["x"]
    else:
        R.close(r, want["r"], mag["r"], 2, "r")
        want2, mag2 = R.layer(r, t["w"], t["b"], None, eps, t["dn"], g_r)  # of the rows as they were kept
        want, mag = {**want, **want2}, {**mag, **mag2}
    R.close(n, want["n"], mag["n"], 64, "n")
    R.close(got["dr"], want["dr"], mag["dr"], 64, "dr")
    R.close(got["dx"], want["dr"], mag["dr"], 64, "dx")
    assert got["dx"].dtype == t["x"].dtype and got["dr"].dtype == r.dtype
    rows = t["x"].numel() // max(t["x"].shape[-1], 1)
    for k in ("dw", "db"):
        if t["w"] is None:
            assert got[k] is None
        else:
            R.close(got[k], want[k], mag[k], 128 + rows, k)
    return r, n, got


@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 16, 31, 33, 64, 100, 128, 255, 256, 257, 264, 1000, 1024, 2047, 2048, 2055, 4096, 4104, 6150,
                               8192, 8200, 12000, 16377, 16384])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_widths(L, D, dtype):
    check(L, make(13, D, dtype, seed=D))
    check(L, make(5, D, dtype, residual=False, affine=D % 2 == 0), dr=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("x32,r32,w32", [(0, 1, 1), (1, 0, 0), (1, 1, 0), (0, 0, 1)])
def test_types(L, dtype, x32, r32, w32):
    pick = lambda k: "f32" if k else dtype  # noqa: E731
    for D in (72, 75, 1203, 1208):
        check(L, make(21, D, dtype, pick(x32), pick(r32), pick(w32)))


@pytest.mark.parametrize("N,D", [(1, 64), (2, 2048), (300, 48), (3000, 40), (5000, 65), (1000, 2056), (700, 9000)])
def test_rows(L, N, D):
    check(L, make(N, D, "bf16", rdtype="f32"))


def test_large_means(L):
    """The variance is that of the differences: a mean of 1000 against a deviation of 1 costs only what the rows' own rounding does."""
    t = make(9, 1500, "f32", mean=1000.0, residual=False)
    check(L, t, dr=False)


def test_rows_that_are_all_the_same(L):
    t = make(4, 96, "f32", residual=False)
    t["x"].fill_(3.0)
    _, n = L.layer_norm_fwd(t["x"], t["w"], t["b"])
    assert torch.equal(n, t["b"].expand(4, 96))


@pytest.mark.parametrize("shift,wide", [(0, 8), (8, 24), (1, 3)])
def test_slices_of_wider_rows(L, shift, wide):
    t = make(30, 80 + wide, "bf16", affine=False)
    w, b = torch.randn(80, device="cuda"), torch.randn(80, device="cuda")
    t.update({k: t[k][:, shift:shift + 80] for k in ("x", "residual", "dn", "dr")}, w=w, b=b)
    check(L, t)
    heads = make(6 * 5, 2 * 48, "bf16", affine=False)
    heads.update({k: heads[k].view(6, 5, 96)[:, :, 48:] for k in ("x", "residual", "dn", "dr")})
    check(L, heads)


def test_residual_in_place(L):
    t = make(20, 300, "bf16", rdtype="f32")
    want, _ = L.layer_norm_fwd(t["x"], t["w"], residual=t["residual"], out_dtype=torch.bfloat16)
    r, _ = L.layer_norm_fwd(t["x"], t["w"], residual=t["residual"], r_out=t["residual"], out_dtype=torch.bfloat16)
    assert r is t["residual"] and torch.equal(r, want)


def test_no_rows(L):
    t = make(0, 64, "f32")
    r, n, g = check(L, t)
    assert n.shape == (0, 64) and not g["dw"].any() and not g["db"].any()


def test_gradients_against_differences(L):
    t = make(4, 37, "f32", seed=2)
    _, _, g = check(L, t)
    args = {k: t[k].double() for k in ("x", "w", "b", "residual")}

    def loss(a):
        out, _ = R.layer(a["x"], a["w"], a["b"], a["residual"])
        return float((out["n"] * t["dn"].double()).sum() + (out["r"] * t["dr"].double()).sum())

    gen = torch.Generator().manual_seed(1)
    for k, name in (("x", "dx"), ("residual", "dr"), ("w", "dw"), ("b", "db")):
        v, h, d = torch.randn(args[k].shape, generator=gen, dtype=torch.float64).cuda(), 1e-5, g[name].double()
        diff = (loss({**args, k: args[k] + h * v}) - loss({**args, k: args[k] - h * v})) / (2 * h)
        assert abs(diff - float((d * v).sum())) <= 2e-5 * (1 + float((d * v).abs().sum())), k


def test_runs_the_same_on_every_call(L):
    t = make(900, 520, "bf16", rdtype="f32")
    a, b = check(L, t), check(L, t)
    assert torch.equal(a[1], b[1]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


@pytest.mark.parametrize("D", [41, 1000, 1203, 3584, 7168])
@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("value", [3.0, 1000.0])
def test_constant_rows_have_no_deviation(L, D, wide, value):
    """Sums of equal whole numbers below 2^24 are exact, and so must their mean be: nothing is left for 1/sqrt(eps) = 316 to raise. Forward the
    bias alone, backward no gradient of the weight, and none of the rows where the cotangent is constant too."""
    t = make(5, D, "f32", residual=False, seed=D)
    t["x"] = torch.full((5, D + wide), value, device="cuda")[:, :D]
    _, n = L.layer_norm_fwd(t["x"], t["w"], t["b"])
    assert torch.equal(n, t["b"].expand(5, D))
    assert not L.layer_norm_bwd(t["x"], t["dn"], t["w"], t["b"])["dw"].any()
    assert not L.layer_norm_bwd(t["x"], torch.full((5, D), 3.0, device="cuda"))["dr"].any()


@pytest.mark.parametrize("D", [41, 1500, 1504])
def test_large_means_to_first_order(L, D):
    """A mean of 1000 against a deviation of 1. The mean is off by the roundings of its sum, d = 22 units (20 additions, 1/D, and itself) of the
    mean magnitude, and the differences by that and no more (they are exact), all of a row's alike; the variance to second order only. So n
    moves by rho d w, and dr by rho^2 d (|mean(m xhat)| + |xhat| |mean m|), beside the 64 units of its own terms. Zeros would not pass."""
    t = make(9, D, "f32", mean=1000.0, residual=False, seed=D)
    _, n = L.layer_norm_fwd(t["x"], t["w"], t["b"])
    got = L.layer_norm_bwd(t["x"], t["dn"], t["w"], t["b"])["dr"]
    want, _ = R.layer(t["x"], t["w"], t["b"], dn=t["dn"])
    r, w, m = t["x"].double(), t["w"].double(), t["dn"].double() * t["w"].double()
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    u = r - mean(r)
    rho = 1 / torch.sqrt(mean(u * u) + 1e-5)
    xhat, unit = u * rho, 2.0 ** -24
    d = 22 * unit * mean(r.abs())
    tol = rho * d * w.abs() + 64 * unit * ((xhat * w).abs() + t["b"].double().abs())
    assert ((n.double() - want["n"]).abs() <= tol).all()
    tol = 64 * unit * rho * (m.abs() + mean(m.abs()) + xhat.abs() * mean((m * xhat).abs()))
    tol = tol + rho * rho * d * (mean(m * xhat).abs() + (xhat.abs() + rho * d) * mean(m).abs())
    assert ((got.double() - want["dr"]).abs() <= tol).all()
    assert (want["dr"].abs() > tol).double().mean() > 0.9


def test_no_rows_of_more_columns_than_an_int_counts(L):
    """Cut off to an int, 2^32 + 16 columns would be 16."""
    x = torch.empty((0, (1 << 32) + 16), device="cuda")
    for f in (lambda: L.layer_norm_fwd(x), lambda: L.layer_norm_bwd(x, x), lambda: L.block_norm_fwd(x)):
        with pytest.raises(L.LatticeError):
            f()
