"""The selective scan on the GPU against the token-by-token 64-bit form, at the sizes where tiles, marks, lanes, groups,
segments, vectors and lengths end.

Units of 2^-24 of the terms' magnitude. A step's decay is off by at most 8 units (the exponential's 2, and dt's 4 times an exponent
that is itself a factor of the decay), its products by 2, so a state is off by 10 times the steps that it remembers, at most
min(T, R) with R = 1/(least dt |A|). A read adds the N terms of its sum, a cotangent as many steps on its side; db, dc, dA
add their channels' or tokens' terms, in parts of at most 16 and then part by part."""
import pytest

import block_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GRADS = ("dx", "ddt", "dA", "db", "dc", "dskip", "dz", "ddt_bias", "dh0")


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


def make(B, T, E, N, G=1, dtype="f32", dtdtype=None, gate=True, skip=True, softplus=True, bias=True, h0=True, lengths=None, wide=False,
         flat=False, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    dt = DT[dtype]
    rows = lambda: n(B, T, 2 * E + 1).to(dt)[:, :, E:2 * E] if wide else n(B, T, E).to(dt)  # noqa: E731
    vec = lambda: n(B, T, G * N + 3).to(dt)[:, :, 1:1 + G * N].unflatten(-1, (G, N)) if wide else n(B, T, G, N).to(dt)  # noqa: E731
    t = {"x": rows(), "z": rows() if gate else None, "b": vec(), "c": vec(),
         "A": -(0.5 + torch.rand((E, N), generator=gen, device="cuda") * 8), "skip": n(E) if skip else None,
         "dt_bias": n(E) - 2 if bias else None, "dt": (n(B, T, E) if softplus else torch.rand((B, T, E), generator=gen, device="cuda") * 0.2
                                                       + 0.01).to(DT[dtdtype or dtype]),
         "softplus": softplus, "h0": n(B, E, N) if h0 else None, "dy": rows(), "dh_T": n(B, E, N) if h0 else None, "lengths": None}
    if not softplus:
        t["dt_bias"] = None
    if flat:
        t["b"], t["c"] = t["b"][:, :, 0], t["c"][:, :, 0]
    if lengths is not None:
        t["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for i, v in enumerate(lengths):
            for k in ("x", "z", "dt", "b", "c", "dy"):
                if t[k] is not None:
                    t[k][i, max(v, 0):] = float("nan")
    return t


def call(L, t):
    args = [t[k] for k in ("x", "dt", "A", "b", "c")]
    how = {k: t[k] for k in ("z", "dt_bias", "softplus", "lengths")}
    marks = L.selective_scan_marks(t["x"], t["A"].shape[1])
    y, h_T = L.selective_scan_fwd(*args, t["skip"], h0=t["h0"], marks=marks, **how)
    got = L.selective_scan_bwd(*args, t["dy"], marks, t["skip"], dh_T=t["dh_T"], **how)
    assert set(got) == set(GRADS)
    got.update(y=y, h_T=h_T)
    return got


def check(L, t):
    got = call(L, t)
    how = {k: t[k] for k in ("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "softplus", "h0", "lengths", "dy", "dh_T")}
    want, mag = R.selective(**how), R.selective(**how, mag=True)
    B, T, E = t["x"].shape
    N = t["A"].shape[1]
    raw = torch.nan_to_num(t["dt"].double(), nan=0.0) + (0 if t["dt_bias"] is None else t["dt_bias"].double())
    d = torch.logaddexp(raw, torch.zeros_like(raw)) if t["softplus"] else raw
    least = float((d.min() if d.numel() else torch.ones(())) * t["A"].abs().min())
    steps = 10 * min(max(T, 1), 1 / max(least, 1e-6))
    units = {"y": steps + N + 16, "h_T": steps, "dh0": steps + N}
    for k in ("dx", "dz", "ddt"):
        units[k] = 2 * steps + 2 * N + 32
    for k in ("db", "dc", "dA", "dskip", "ddt_bias"):
        units[k] = 2 * steps + 2 * N + 64 + max(E, T * B) // 16
    for k in GRADS + ("y", "h_T"):
        absent = {"dskip": "skip", "dz": "z", "ddt_bias": "dt_bias"}.get(k)
        if absent and t[absent] is None:
            assert got[k] is None
        else:
            R.close(got[k], want[k], mag[k], units[k], k)
    return got


@pytest.mark.parametrize("B,T,E,N,G", [(1, 1, 1, 1, 1), (2, 16, 64, 16, 1), (3, 17, 65, 16, 1), (1, 33, 6, 4, 2), (2, 50, 130, 13, 2),
                                       (1, 40, 41, 8, 1), (2, 24, 33, 32, 1), (1, 21, 18, 64, 3), (1, 19, 20, 128, 1), (1, 18, 9, 100, 1),
                                       (2, 31, 48, 3, 4), (1, 15, 257, 7, 1), (2, 9, 34, 20, 2), (1, 8, 12, 33, 1)])
@pytest.mark.parametrize("gate", [True, False])
def test_sizes(L, B, T, E, N, G, gate):
    check(L, make(B, T, E, N, G, gate=gate, skip=gate))


@pytest.mark.parametrize("dtype,dtdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("wide", [False, True])
def test_types_and_slices(L, dtype, dtdtype, wide):
    check(L, make(2, 37, 66, 16, 1, dtype, dtdtype, wide=wide))
    check(L, make(2, 20, 66, 10, 2, dtype, dtdtype, wide=wide, h0=False))


def test_plain_steps_and_no_bias(L):
    check(L, make(2, 30, 40, 16, softplus=False))
    check(L, make(2, 30, 40, 16, bias=False, skip=False, gate=False, h0=False))


@pytest.mark.parametrize("B,T,E,N,G", [(1, 700, 8, 16, 1), (1, 1000, 20, 16, 2), (2, 515, 10, 5, 1), (1, 1300, 70, 32, 1), (1, 400, 9, 64, 1),
                                       (1, 270, 4, 128, 2), (1, 800, 4, 128, 2)])
def test_few_channels_of_long_sequences(L, B, T, E, N, G):
    """The time axis is split (from three segments on: two would cost as much as one)."""
    assert T < 384 or L.lib().lattice_selective_scan_workspace_bytes(B, T, E, N, G, 0) > 0
    check(L, make(B, T, E, N, G))
    check(L, make(B, T, E, N, G, "bf16", lengths=[T * 2 // 3] * B))


@pytest.mark.parametrize("B,E", [(160, 64), (310, 128), (75, 256)])
def test_many_sequences(L, B, E):
    """More CTAs than the device has SMs: both widths of a lane's share."""
    t = make(B, 18, E, 16, dtype="bf16")
    got = call(L, t)
    for lo in (0, B - 2):
        part = {k: v[lo:lo + 2] if isinstance(v, torch.Tensor) and v.dim() and v.shape[0] == B and k not in ("A", "skip", "dt_bias") else v
                for k, v in t.items()}
        one = check(L, part)
        for k in ("dx", "ddt", "dz", "dh0", "h_T", "y"):
            R.close(one[k], got[k][lo:lo + 2].double(), got[k][lo:lo + 2].double().abs() + got[k].double().abs().mean(),
                    2000 + 2 ** 17 * (one[k].dtype != torch.float32), k)  # two sums in another order, each rounded


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths(L, dtype):
    lens = [0, 1, 7, 8, 9, 16, 33, 50, 70, -3]
    got = check(L, make(10, 50, 36, 16, 2, dtype, lengths=lens))
    for i, n in enumerate(lens):
        n = min(max(n, 0), 50)
        for k in ("y", "dx", "ddt", "dz", "db", "dc"):
            assert not got[k][i, n:].any(), k


def test_no_tokens(L):
    t = make(2, 0, 8, 16)
    got = check(L, t)
    assert torch.equal(got["h_T"], t["h0"]) and torch.equal(got["dh0"], t["dh_T"]) and not got["dA"].any()


def test_long_memory(L):
    """Decays near 1: an error with a mean would grow with the steps remembered. 4000 steps of dt |A| = 2e-4 to 8e-3: the state's relative
    error is held to what random errors of half a step in the decay and the sum give, 2^-24 sqrt(1/(2 dt |A|)) each, and 6 times that."""
    B, T, E, N = 1, 4000, 32, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, b, c = n(B, T, E), n(B, T, N), n(B, T, N)
    A = -(torch.arange(1, N + 1, device="cuda").float() * 0.5).expand(E, N).contiguous()
    dt = torch.linspace(4e-4, 1e-3, E, device="cuda").expand(B, T, E) * (1 + 0.2 * torch.rand((B, T, E), generator=gen, device="cuda"))
    dt = dt.contiguous()
    _, h = L.selective_scan_fwd(x, dt, A, b, c, softplus=False)
    want = R.selective(x, dt, A, b, c, softplus=False)["h_T"]
    rel = float((h.double() - want).norm() / want.norm())
    assert rel <= 6 * 2 * 2.0 ** -24 * (1 / (2 * 2e-4)) ** 0.5, rel


def test_in_pieces_and_by_single_tokens(L):
    t = make(3, 40, 33, 16, 1, "bf16")
    how = {"skip": t["skip"], "dt_bias": t["dt_bias"]}
    at = lambda lo, hi: [t["x"][:, lo:hi], t["dt"][:, lo:hi], t["A"], t["b"][:, lo:hi], t["c"][:, lo:hi]]  # noqa: E731
    y, end = L.selective_scan_fwd(*at(0, 40), h0=t["h0"], z=t["z"], **how)
    h = t["h0"].clone()
    first, h = L.selective_scan_fwd(*at(0, 17), h0=h, h_out=h, z=t["z"][:, :17], **how)  # in place
    parts = [first]
    for k in range(17, 40):
        one = [v[:, 0] if v.dim() > 2 else v for v in at(k, k + 1)]
        parts.append(L.selective_step(h, *one, z=t["z"][:, k], **how)[:, None])
    want = R.selective(t["x"], t["dt"], t["A"], t["b"], t["c"], z=t["z"], h0=t["h0"], **how)
    mag = R.selective(t["x"], t["dt"], t["A"], t["b"], t["c"], z=t["z"], h0=t["h0"], mag=True, **how)
    for got, hh in ((y, end), (torch.cat(parts, 1), h)):
        R.close(got, want["y"], mag["y"], 432, "y")  # 10 * 40 + 16 + 16
        R.close(hh, want["h_T"], mag["h_T"], 400, "h_T")


@pytest.mark.parametrize("dtype,dtdtype,E,N,G", [("f32", "f32", 5, 1, 1), ("bf16", "f32", 66, 16, 1), ("f16", "f16", 12, 13, 3),
                                                 ("bf16", "bf16", 7, 64, 1), ("f32", "f32", 3, 128, 1), ("bf16", "bf16", 40, 30, 2),
                                                 ("f32", "f32", 9, 4, 1), ("f32", "f32", 9, 8, 1)])
def test_step(L, dtype, dtdtype, E, N, G):
    t = make(5, 1, E, N, G, dtype, dtdtype)
    out, before = torch.empty_like(t["h0"]), t["h0"].clone()
    y = L.selective_step(t["h0"], t["x"][:, 0], t["dt"][:, 0], t["A"], t["b"][:, 0], t["c"][:, 0], t["skip"], z=t["z"][:, 0],
                         dt_bias=t["dt_bias"], h_out=out)
    how = {k: t[k] for k in ("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "h0")}
    want, mag = R.selective(**how), R.selective(**how, mag=True)
    R.close(y, want["y"][:, 0], mag["y"][:, 0], 10 + N + 16, "y")
    R.close(out, want["h_T"], mag["h_T"], 10, "h")
    assert torch.equal(before, t["h0"])


def test_step_sizes_at_their_ends(L):
    """dt_raw so far down that dt is 0 and the state stays; so far up that softplus is the identity and the old state is gone."""
    t = make(2, 3, 4, 16)
    t["dt_bias"] = None
    t["dt"][:, 0], t["dt"][:, 1], t["dt"][:, 2] = -200.0, -float("inf"), 200.0
    y, h = L.selective_scan_fwd(t["x"], t["dt"], t["A"], t["b"], t["c"], h0=t["h0"])
    _, kept = L.selective_scan_fwd(t["x"][:, :2], t["dt"][:, :2].contiguous(), t["A"], t["b"][:, :2], t["c"][:, :2], h0=t["h0"])
    assert torch.equal(kept, t["h0"])
    want = 200.0 * t["x"][:, 2, :, None].double() * t["b"][:, 2].double()
    R.close(h, want, want.abs() + 1e-30, 8, "h")


def test_gradients_against_differences(L):
    t = make(2, 11, 6, 5, 2, lengths=[11, 6], seed=4)
    for k in ("x", "z", "dt", "b", "c", "dy"):
        t[k] = torch.nan_to_num(t[k])
    got = check(L, t)
    names = ("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "h0")
    args = {k: t[k].double() for k in names}

    def loss(a):
        out = R.selective(**a, lengths=t["lengths"])
        return float((out["y"] * t["dy"].double()).sum() + (out["h_T"] * t["dh_T"].double()).sum())

    gen = torch.Generator().manual_seed(1)
    for k in names:
        v, h, g = torch.randn(args[k].shape, generator=gen, dtype=torch.float64).cuda(), 1e-5, got["d" + k].double()
        diff = (loss({**args, k: args[k] + h * v}) - loss({**args, k: args[k] - h * v})) / (2 * h)
        assert abs(diff - float((g * v).sum())) <= 2e-5 * (1 + float((g * v).abs().sum())), k


def test_runs_the_same_on_every_call(L):
    for t in (make(3, 90, 130, 16, dtype="bf16", lengths=[90, 3, 41]), make(1, 900, 20, 16)):
        a, b = call(L, t), call(L, t)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_without_marks_and_marks_alone(L):
    t = make(2, 40, 32, 16)
    args = [t[k] for k in ("x", "dt", "A", "b", "c")]
    y, h = L.selective_scan_fwd(*args, h0=t["h0"])
    marks = L.selective_scan_marks(t["x"], 16)
    y2, h2 = L.selective_scan_fwd(*args, h0=t["h0"], marks=marks)
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(marks[:, 0], t["h0"])


@pytest.mark.parametrize("T", [900, 5000])
def test_state_in_place_over_segments(L, T):
    """The final state over the initial one, which all segments' entering states need: the same as into another place."""
    t = make(1, T, 24, 16)
    args, how = [t[k] for k in ("x", "dt", "A", "b", "c")], {"skip": t["skip"], "z": t["z"], "dt_bias": t["dt_bias"] - 5}  # long memory
    assert L.lib().lattice_selective_scan_workspace_bytes(1, T, 24, 16, 1, 0) > 0
    y, h = L.selective_scan_fwd(*args, h0=t["h0"], **how)
    state = t["h0"].clone()
    y2, h2 = L.selective_scan_fwd(*args, h0=state, h_out=state, **how)
    assert h2 is state and torch.equal(y, y2) and torch.equal(h, h2)


def test_growing_states_over_segments(L):
    """A > 0, whose growth over a segment is past the largest number, on states and cotangents that are 0 there."""
    t = make(1, 900, 12, 16, softplus=False, h0=False)
    t["A"] = -t["A"]
    t["x"][:, :-5], t["dy"][:, 5:] = 0.0, 0.0
    got = call(L, t)
    how = {k: t[k] for k in ("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "softplus", "h0", "lengths", "dy", "dh_T")}
    want, mag = R.selective(**how), R.selective(**how, mag=True)
    for k in ("y", "h_T", "dx", "dz", "ddt", "db", "dc", "dA"):  # 5 steps remembered: 2 * 10 * 5 + 2 * 16 + 64 + 900 / 16
        assert torch.isfinite(got[k]).all(), k
        R.close(got[k], want[k], mag[k], 253, k)


def test_most_channels(L):
    """The largest E: one token of 2^30 channels with one state each, some 60 GB, whose gradients per channel are checked at both ends and
    in the middle."""
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    E, N = 1 << 30, 1
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda").normal_(generator=gen)  # noqa: E731
    t = {"x": n(1, 1, E), "dt": n(1, 1, E), "A": n(E, N, dtype=torch.float32).abs_().neg_(), "b": n(1, 1, N), "c": n(1, 1, N),
         "skip": n(E, dtype=torch.float32), "dt_bias": n(E, dtype=torch.float32), "dy": n(1, 1, E)}
    args = [t[k] for k in ("x", "dt", "A", "b", "c")]
    marks = L.selective_scan_marks(t["x"], N)
    y, h_T = L.selective_scan_fwd(*args, t["skip"], dt_bias=t["dt_bias"], marks=marks)
    got = L.selective_scan_bwd(*args, t["dy"], marks, t["skip"], dt_bias=t["dt_bias"])
    got.update(y=y, h_T=h_T)
    for lo in (0, E // 2, E - 1000):
        of = {k: slice(lo, lo + 1000) for k in ("x", "dt", "dy", "y", "dx", "ddt", "A", "dA", "skip", "dskip", "dt_bias", "ddt_bias", "h_T", "dh0")}
        cut = lambda k, v: v[of[k]] if v.shape[0] == E else v[..., of[k], :] if k in ("h_T", "dh0") else v[..., of[k]]  # noqa: E731
        how = {k: cut(k, v) if k in of else v for k, v in t.items()}
        want, mag = R.selective(**how), R.selective(**how, mag=True)
        for k in ("y", "h_T", "dx", "ddt", "dA", "dskip", "ddt_bias", "dh0"):  # one step remembered: 2 * 10 + 2 * 1 + 64
            R.close(cut(k, got[k]), want[k], mag[k], 86, k)
    del t, args, marks, y, h_T, got, how, want, mag
    torch.cuda.empty_cache()


def test_more_segments_than_a_cta_goes_through(L):
    """More than 32 segments, whose entering states and cotangents a launch of its own joins: both directions against the 64-bit form, with
    states from before, cotangents from behind, an end inside a segment, and a memory of several segments (dt |A| from 2.5e-3 to 0.085)."""
    B, T, E, N = 2, 3000, 24, 16
    t = make(B, T, E, N, gate=False, softplus=False, lengths=[T, 1111], seed=6)
    t["dt"] = 0.05 + (t["dt"] - 0.01) * 0.25
    t["A"], t["h0"], t["dh_T"] = t["A"] / 10, 30 * t["h0"], 30 * t["dh_T"]
    row = E * N + E  # a segment's states and sum of steps; backward as much for dA's parts, 2 E for two sums, and db's and dc's per CTA of 16
    ws = L.lib().lattice_selective_scan_workspace_bytes
    assert ws(B, T, E, N, 1, 0) > 4 * B * 32 * row and ws(B, T, E, N, 1, 1) > 4 * (B * 32 * (2 * row + E) + 2 * B * T * 2 * N)
    got = check(L, t)
    how = {k: t[k] for k in ("x", "dt", "A", "b", "c", "skip", "z", "dt_bias", "softplus", "h0", "lengths", "dy", "dh_T")}
    mag = R.selective(**how, mag=True)
    # the bounds tell a state or cotangent that was not handed on: 8 segments of 64 tokens from where it enters
    without, at = R.selective(**{**how, "h0": None}), slice(512, 520)
    with pytest.raises(AssertionError):
        R.close(got["y"][:1, at], without["y"][:1, at], mag["y"][:1, at], 5000 + N + 16, "y")
    without, at = R.selective(**{**how, "dh_T": None}), slice(T - 520, T - 512)
    with pytest.raises(AssertionError):
        R.close(got["dx"][:1, at], without["dx"][:1, at], mag["dx"][:1, at], 10000 + 2 * N + 32, "dx")
