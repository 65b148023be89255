"""The short convolution on the GPU against the 64-bit form, at the sizes where runs, vectors, taps, states and lengths end.

Units of 2^-24 of the terms' magnitude: K + 1 multiply-adds, and for silu an exponential and a reciprocal (2 units each),
whose argument carries the sum's error on (at most |v| + 4 units of |y|, and less for large |v|, where the logistic function is flat):
16 + 2 K. The gradients sum K or the tokens' terms more; a run's tokens one by one, then the runs."""
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


def make(B, T, C, K, dtype="f32", wdtype=None, state=True, lengths=None, wide=0, shift=0, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    dt = DT[dtype]

    def rows():
        if not wide:
            return n(B, T, C).to(dt)
        return n(B, T, C + wide).to(dt)[:, :, shift:shift + C]

    t = {"x": rows(), "w": n(C, K).to(DT[wdtype or dtype]), "bias": n(C).to(DT[wdtype or dtype]), "dy": rows(), "lengths": None,
         "state": n(B, K - 1, C).to(dt) if state else None, "dstate_out": n(B, K - 1, C).to(dt)}
    if lengths is not None:
        t["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for b, v in enumerate(lengths):
            t["x"][b, max(v, 0):] = float("nan")
            t["dy"][b, max(v, 0):] = float("nan")
    return t


def check(L, t, act="silu", bias=True, dstate=True):
    b = t["bias"] if bias else None
    ds = t["dstate_out"] if dstate else None
    how = dict(act=act, state=t["state"], lengths=t["lengths"])
    y, state = L.short_conv_fwd(t["x"], t["w"], b, **how)
    got = L.short_conv_bwd(t["x"], t["w"], t["dy"], b, dstate_out=ds, **how)
    want, mag = R.conv(t["x"], t["w"], b, dy=t["dy"], dstate_out=ds, **how)
    B, T, C = t["x"].shape
    K = t["w"].shape[1]
    R.close(y, want["y"], mag["y"], 16 + 2 * K, "y")
    assert torch.equal(state.double(), want["state"])
    R.close(got["dx"], want["dx"], mag["dx"], 32 + 4 * K, "dx")
    sums = 32 + 4 * K + min(T, 1024) + B * T // 64
    R.close(got["dw"], want["dw"], mag["dw"], sums, "dw")
    if bias:
        R.close(got["dbias"], want["dbias"], mag["dbias"], sums, "dbias")
    else:
        assert got["dbias"] is None
    if t["state"] is None:
        assert got["dstate"] is None
    else:
        R.close(got["dstate"], want["dstate"], mag["dstate"], 32 + 4 * K, "dstate")
    return y, state, got


@pytest.mark.parametrize("K", range(1, 9))
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_taps_and_types(L, K, dtype):
    check(L, make(2, 70, 40, K, dtype, seed=K))


@pytest.mark.parametrize("B,T,C,K", [(1, 1, 1, 4), (1, 1, 8, 4), (3, 2, 5, 4), (2, 3, 16, 8), (2, 7, 33, 3), (1, 129, 24, 4), (2, 65, 1030, 4),
                                     (1, 1000, 4, 2), (5, 31, 2048, 4), (1, 3000, 2, 5), (130, 9, 64, 4)])
def test_sizes(L, B, T, C, K):
    check(L, make(B, T, C, K, "bf16", "f32"))
    check(L, make(B, T, C, K, "f32", state=False), act="none", bias=False, dstate=False)


@pytest.mark.parametrize("dtype,wide,shift", [("bf16", 8, 8), ("bf16", 4, 4), ("bf16", 3, 1), ("f32", 2, 2), ("f32", 4, 0), ("f16", 16, 3)])
def test_slices_of_wider_rows(L, dtype, wide, shift):
    check(L, make(2, 45, 32, 4, dtype, wide=wide, shift=shift))


def test_batch_and_token_axes_in_another_order(L):
    t = make(3, 20, 16, 4, "bf16")
    for k in ("x", "dy"):
        t[k] = t[k].transpose(0, 1).contiguous().transpose(0, 1)
    check(L, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
def test_lengths(L, dtype, state):
    # none, fewer than the taps, a run's end, the whole, more, and less than nothing
    t = make(9, 70, 24, 4, dtype, state=state, lengths=[0, 1, 2, 3, 33, 64, 70, 90, -5])
    y, _, g = check(L, t)
    for b, n in enumerate([0, 1, 2, 3, 33, 64, 70, 70, 0]):
        assert not y[b, n:].any() and not g["dx"][b, n:].any()


def test_no_tokens(L):
    t = make(2, 0, 8, 4, "f32")
    y, state, g = check(L, t)
    assert torch.equal(state, t["state"]) and not g["dw"].any()


def test_in_pieces_and_by_single_tokens(L):
    t = make(3, 40, 24, 4, "bf16", seed=3)
    y, end = L.short_conv_fwd(t["x"], t["w"], t["bias"], state=t["state"])
    s = t["state"].clone()
    first, s = L.short_conv_fwd(t["x"][:, :17], t["w"], t["bias"], state=s, state_out=s)  # in place
    parts = [first]
    for k in range(17, 40):
        parts.append(L.short_conv_step(s, t["x"][:, k], t["w"], t["bias"])[:, None])
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(s, end)


@pytest.mark.parametrize("dtype,C", [("f32", 5), ("bf16", 64), ("f16", 12), ("bf16", 33)])
@pytest.mark.parametrize("K", [1, 2, 4, 7])
def test_step(L, dtype, C, K):
    t = make(7, 1, C, K, dtype, seed=K)
    x = t["x"][:, 0]
    out = torch.empty_like(t["state"])
    before = t["state"].clone()
    y = L.short_conv_step(t["state"], x, t["w"], t["bias"], act="none", state_out=out)
    want, mag = R.conv(t["x"], t["w"], t["bias"], "none", t["state"])
    R.close(y, want["y"][:, 0], mag["y"][:, 0], 16 + 2 * K, "y")
    assert torch.equal(out.double(), want["state"]) and torch.equal(before, t["state"])


def test_infinities_stay_with_the_tokens_that_see_them(L):
    t = make(1, 30, 8, 3, "f32", state=False)
    t["x"][0, 10, 2] = float("inf")
    y, _ = L.short_conv_fwd(t["x"], t["w"], t["bias"], act="none")
    bad = ~torch.isfinite(y)
    assert sorted(bad.nonzero()[:, 1].tolist()) == [10, 11, 12] and set(bad.nonzero()[:, 2].tolist()) == {2}


def test_gradients_against_differences(L):
    t = make(2, 12, 6, 4, "f32", seed=5, lengths=[12, 7])
    for k in ("x", "dy"):
        t[k] = torch.nan_to_num(t[k])
    _, _, g = check(L, t)

    def loss(x, w, bias, state):
        out, _ = R.conv(x, w, bias, "silu", state, t["lengths"])
        return float((out["y"] * t["dy"].double()).sum() + (out["state"] * t["dstate_out"].double()).sum())

    args = [t[k].double() for k in ("x", "w", "bias", "state")]
    gen = torch.Generator().manual_seed(1)
    for k, name in enumerate(("dx", "dw", "dbias", "dstate")):
        v = torch.randn(args[k].shape, generator=gen, dtype=torch.float64).cuda()
        h = 1e-5
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * v, args[k] - h * v
        diff, want = (loss(*up) - loss(*down)) / (2 * h), float((g[name].double() * v).sum())
        assert abs(diff - want) <= 1e-5 * (1 + float((g[name].double() * v).abs().sum())), name


def test_runs_the_same_on_every_call(L):
    t = make(3, 700, 130, 4, "bf16", lengths=[700, 3, 411])
    a, b = (check(L, t) for _ in range(2))
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])
