"""The gated linear recurrence on the GPU against the token-by-token 64-bit form, at the
sizes where tiles, runs, clusters, vectors and lengths end."""
import itertools
import math

import pytest

import gated_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


def make(B, T, H, d, dtype="f32", zdtype=None, gate="logit", head=False, seed=0, mean=2.0, lengths=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    z = n(B, T, H) if head else n(B, T, H, d)
    z = 1.2 * z + mean
    if gate == "value":
        z = 2 * torch.sigmoid(z) - 1 if mean < 1 else torch.sigmoid(z)
    t = {"x": n(B, T, H, d).to(DT[dtype]), "z": z.to(DT[zdtype or dtype]), "h0": n(B, H, d), "dy": n(B, T, H, d).to(DT[dtype]),
         "dh_T": n(B, H, d), "lengths": None}
    if lengths is not None:
        t["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for b, v in enumerate(lengths):
            for k in ("x", "z", "dy"):
                t[k][b, max(v, 0):] = float("nan")
    return t


def both(L, t, gate="logit", write="leaky", tau=1.0, h0=True, dh_T=True):
    kw = dict(gate=gate, write=write, tau=tau, lengths=t["lengths"])
    h = t["h0"] if h0 else None
    k = t["dh_T"] if dh_T else None
    marks = L.gated_scan_marks(t["x"])
    y, h_T = L.gated_scan_fwd(t["x"], t["z"], h, marks=marks, **kw)
    got = L.gated_scan_bwd(t["x"], t["z"], t["dy"], marks, dh_T=k, **kw)
    got.update(y=y, h_T=h_T)
    lens = None if t["lengths"] is None else t["lengths"].tolist()
    ref = R.scan(t["x"], t["z"], h, gate, write, tau, lens, t["dy"], k)
    for name in ("y", "h_T", "dx", "dz", "dh0"):
        R.check(got[name], ref, name)
    assert got["y"].dtype == t["x"].dtype and got["dz"].dtype == t["z"].dtype and got["dx"].dtype == t["x"].dtype
    return got


SHAPES = [(1, 1, 1, 1), (2, 7, 1, 5), (1, 8, 2, 16), (2, 63, 1, 37), (1, 64, 3, 16), (3, 65, 2, 64), (2, 127, 1, 130),
          (1, 513, 2, 32), (1, 1537, 1, 66), (33, 129, 5, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,zdtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_shapes_and_types(L, shape, dtype, zdtype):
    both(L, make(*shape, dtype=dtype, zdtype=zdtype, seed=sum(shape)))


@pytest.mark.parametrize("gate,write,tau", list(itertools.product(["value"], ["plain", "leaky", "unit"], [1.0]))
                         + list(itertools.product(["logit"], ["plain", "leaky", "unit"], [1.0, 0.0625, 2.5])))
@pytest.mark.parametrize("head", [False, True])
def test_forms(L, gate, write, tau, head):
    both(L, make(2, 150, 3, 32, gate=gate, head=head, seed=3), gate, write, tau)
    both(L, make(2, 150, 3, 32, dtype="bf16", zdtype="f32", gate=gate, head=head, seed=4, mean=0.0), gate, write, tau)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,zdtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_head_gates(L, d, dtype, zdtype):
    both(L, make(2, 131, 5, d, dtype=dtype, zdtype=zdtype, head=True, seed=d), write="unit")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,d", [(2, 16), (4, 16), (10, 16), (2, 32), (6, 32), (2, 64), (4, 64), (12, 64), (2, 128), (16, 128)])
def test_head_gates_in_16_bits(L, H, d, dtype):
    """An even number of heads: a token's gates are whole words, which are copied as such. Gates
    that start on an odd element, or rows an odd number of elements apart, are copied one by one."""
    both(L, make(2, 131, H, d, dtype=dtype, head=True, seed=H + d), write="unit")
    t = make(3, 77, H, d, dtype=dtype, head=True, seed=H, lengths=[77, 0, 34])
    want = both(L, t, tau=0.25)
    for pad, first in ((0, 1), (1, 0), (2, 1), (4, 2), (6, 0)):  # wider rows, in words or not
        wide = torch.full((3, 77, H + pad + first), float("nan"), dtype=DT[dtype], device="cuda")
        moved = dict(t, z=wide[:, :, first:first + H])
        moved["z"].copy_(t["z"])
        got = both(L, moved, tau=0.25)
        assert all(torch.equal(got[k], want[k]) for k in want), (pad, first)


@pytest.mark.parametrize("lengths", [[0, 0, 0], [0, 1, 200], [64, 63, 65], [200, 128, 7], [-3, 199, 9999]], ids=str)
@pytest.mark.parametrize("head", [False, True])
def test_padded_batches(L, lengths, head):
    got = both(L, make(3, 200, 2, 32, dtype="bf16", zdtype="f32", head=head, seed=9, lengths=lengths), write="unit")
    for b, v in enumerate(lengths):
        for k in ("y", "dx", "dz"):
            assert (got[k][b, max(v, 0):] == 0).all()


def test_long_sequence_of_few_channels_spreads_over_a_cluster(L):
    both(L, make(1, 6000, 1, 24, mean=6.0, seed=5), write="unit")
    both(L, make(1, 6000, 1, 24, mean=6.0, seed=5, lengths=[4321]), write="leaky", tau=0.25)


@pytest.mark.parametrize("dtype,zdtype,d,head", [("bf16", "bf16", 37, False), ("f16", "f32", 64, False),
                                                 ("bf16", "bf16", 64, True), ("f32", "f32", 64, True)])
def test_long_sequences_in_clusters_above_the_portable_size(L, dtype, zdtype, d, head):
    both(L, make(2, 4700, 1, d, dtype=dtype, zdtype=zdtype, head=head, mean=5.0, seed=11, lengths=[4700, 2063]), write="unit")


@pytest.mark.parametrize("dtype,zdtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("B,T,H,d", [(2, 700, 1, 63), (1, 333, 1, 65), (2, 130, 13, 5), (3, 260, 3, 43), (5, 40, 1, 1)])
def test_odd_channels(L, B, T, H, d, dtype, zdtype):
    both(L, make(B, T, H, d, dtype=dtype, zdtype=zdtype, seed=T + d, mean=1.0), write="unit", tau=0.25)
    lengths = [T - 1 - 17 * b for b in range(B)]
    both(L, make(B, T, H, d, dtype=dtype, zdtype=zdtype, seed=T, lengths=lengths))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,head", [(32, False), (33, False), (64, True), (7, False)])
def test_arrays_that_start_anywhere(L, d, head, dtype):
    """What stands around the rows is neither read into them nor written."""
    B, T, H = 2, 150, 1
    t = make(B, T, H, d, dtype=dtype, head=head, seed=31)
    want = both(L, t)
    for k in ("x", "z", "dy"):
        wide = torch.full((B * T * t[k][0, 0].numel() + 9,), float("nan"), dtype=t[k].dtype, device="cuda")
        for off in (1, 3):
            wide[:] = float("nan")
            part = wide[off:off + t[k].numel()].view(t[k].shape)
            part.copy_(t[k])
            moved = dict(t)
            moved[k] = part
            got = both(L, moved)
            # a head's dz is a sum of products, of which the kernel for such rows may round one less
            assert all(torch.equal(got[n], want[n]) for n in want if n != "dz" or not head)
    for off in (0, 1, 2, 5):
        room = torch.full((t["x"].numel() + 16,), 7.0, dtype=t["x"].dtype, device="cuda")
        y = room[off:off + t["x"].numel()].view(t["x"].shape)
        L.gated_scan_fwd(t["x"], t["z"], t["h0"], y=y, write="leaky")
        assert torch.equal(y, want["y"]) and (room[:off] == 7).all() and (room[off + y.numel():] == 7).all()


def test_large_clusters_on_two_streams_at_once(L):
    """Clusters of many CTAs, launched side by side: each call's results are its own."""
    ts = [make(1, 5000, 1, d, dtype="bf16", mean=4.0, seed=40 + d) for d in (40, 64)]
    want = []
    for t in ts:
        marks = L.gated_scan_marks(t["x"])
        y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"], marks=marks)
        want.append((y, h, L.gated_scan_bwd(t["x"], t["z"], t["dy"], marks)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = [[], []]
    for _ in range(10):
        for k, (t, s) in enumerate(zip(ts, streams)):
            with torch.cuda.stream(s):
                marks = L.gated_scan_marks(t["x"])
                y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"], marks=marks)
                got[k].append((y, h, L.gated_scan_bwd(t["x"], t["z"], t["dy"], marks)))
    torch.cuda.synchronize()
    for k in range(2):
        for y, h, g in got[k]:
            assert torch.equal(y, want[k][0]) and torch.equal(h, want[k][1])
            assert all(torch.equal(g[n], want[k][2][n]) for n in g)


def test_no_initial_state_and_no_final_cotangent(L):
    both(L, make(2, 100, 1, 20, seed=6), h0=False, dh_T=False)


def test_no_tokens(L):
    t = make(2, 0, 3, 16)
    y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"])
    assert y.shape == (2, 0, 3, 16) and torch.equal(h, t["h0"])
    g = L.gated_scan_bwd(t["x"], t["z"], t["dy"], L.gated_scan_marks(t["x"]), dh_T=t["dh_T"])
    assert torch.equal(g["dh0"], t["dh_T"])


def test_slices_of_wider_rows(L):
    B, T, H, d = 2, 90, 2, 32
    t = make(B, T, H, d, dtype="bf16", seed=7)
    want = both(L, t)
    for pad in (0, 1, 8):  # 1: rows that vectors cannot read
        wide = torch.full((B, T, 3 * H * d + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        for k, name in enumerate(("x", "z", "dy")):
            v = wide[:, :, k * H * d + pad:(k + 1) * H * d + pad].unflatten(-1, (H, d))
            v.copy_(t[name])
            t[name] = v
        got = both(L, t)
        for k in want:
            assert torch.equal(got[k], want[k]), (pad, k)
    # time-major storage, and one row shared by the batch
    t = make(B, T, H, d, seed=8)
    want = both(L, t)
    t["x"], t["z"], t["dy"] = (t[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "z", "dy"))
    got = both(L, t)
    assert all(torch.equal(got[k], want[k]) for k in want)
    t["x"] = t["x"][:1].expand(B, T, H, d)
    both(L, t)


def test_misaligned_arrays(L):
    B, T, H, d = 2, 70, 1, 32
    t = make(B, T, H, d, dtype="bf16", zdtype="f32", seed=10)
    want = both(L, t)
    for k in ("x", "z", "h0", "dy", "dh_T"):
        flat = torch.empty(t[k].numel() + 1, dtype=t[k].dtype, device="cuda")
        v = flat[1:].view(t[k].shape)
        v.copy_(t[k])
        t[k] = v
    got = both(L, t)
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_in_place_state_and_pieces(L):
    t = make(2, 300, 2, 32, seed=11)
    y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"])
    s = t["h0"].clone()
    parts = []
    for lo, hi in ((0, 1), (1, 130), (130, 130), (130, 300)):
        yp, out = L.gated_scan_fwd(t["x"][:, lo:hi], t["z"][:, lo:hi], s, h_out=s)
        assert out is s
        parts.append(yp)
    ref = R.scan(t["x"], t["z"], t["h0"], "logit", "leaky", 1.0)
    R.check(torch.cat(parts, 1), ref, "y")
    R.check(s, ref, "h_T")


def test_extreme_gates(L):
    inf = float("inf")
    t = make(1, 70, 1, 16, seed=12)
    t["z"][0, 10] = -inf   # forget everything
    t["z"][0, 20] = inf    # keep everything
    t["z"][0, 30] = 200.0
    t["z"][0, 40] = -200.0
    for write, tau in itertools.product(("plain", "leaky", "unit"), (1.0, 0.125)):
        kw = dict(write=write, tau=tau)
        marks = L.gated_scan_marks(t["x"])
        y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"], marks=marks, **kw)
        g = L.gated_scan_bwd(t["x"], t["z"], t["dy"], marks, dh_T=t["dh_T"], **kw)
        for v in (y, h, g["dx"], g["dz"], g["dh0"]):
            assert torch.isfinite(v).all()
        ref = R.scan(t["x"], t["z"], t["h0"], "logit", write, tau)
        R.check(y, ref, "y")
        other = t["dy"].clone()
        other[0, 10:] += 1.0
        g2 = L.gated_scan_bwd(t["x"], t["z"], other, marks, dh_T=3 * t["dh_T"], **kw)
        assert torch.equal(g["dh0"], g2["dh0"])  # nothing passes a gate of 0
        assert (g["dz"][0, [10, 20]] == 0).all()
    t = make(1, 70, 1, 16, seed=12, gate="value")
    t["z"][0, 10], t["z"][0, 20], t["z"][0, 30] = 0.0, 1.0, -1.0
    for write in ("plain", "leaky", "unit"):
        both(L, t, "value", write)


@pytest.mark.parametrize("tau", [0.001, 0.0625, 0.125, 0.3, 0.5, 0.75, 0.999, 1.0, 1.5, 2.5, 10.0])
def test_gates_alone(L, tau):
    """a, 1 - a and sqrt(1 - a^2) as one step from h = 1, x = 0, or from h = 0, x = 1, gives them.
    With e = 2^-24: exp(-|z|) is off by 2 + 1.5 |z| (its argument's rounding); the polynomial's
    coefficients and its sum by 14 each, with alternating terms of up to 14 times the value; each
    halving of tau is a squaring, which leaves 1 - a's relative error as it is and adds 2, and
    doubles a's. z < 0 has the factor exp(tau z): 2 + 1.5 tau |z|, its 1 - exp() within 12. In all
    1 - a is off by 45 + 2 s + 3 (1 + tau) |z| of itself, a by that of 1 - a and one rounding where a > 1/2,
    else by 2^s times that of itself. tau = 1 has no polynomial: a = r (2 - (1 + t) r) rounds 1 + t, the
    bracket and the product, 3 in place of that one rounding (r's own error enters squared)."""
    z = torch.cat([torch.linspace(-30, 30, 4001), torch.tensor([0.0, -0.0, 1e-20, -1e-20, 87.0, 100.0, -100.0, -1000.0, 1000.0]),
                   torch.logspace(-9, 1.5, 2000), -torch.logspace(-9, 1.5, 2000)]).cuda().view(1, 1, -1)
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    out = [torch.empty_like(z) for _ in range(3)]
    for (h, x, write), o in zip(((one, zero, "plain"), (zero, one, "leaky"), (zero, one, "unit")), out):
        L.gated_step(h, x, z, gate="logit", write=write, tau=tau, h_out=o)
    w = tau * torch.nn.functional.logsigmoid(z.double())
    a, q = w.exp(), -torch.expm1(w)
    s = max(0, math.ceil(math.log2(tau)))
    off = (45 + 2 * s + 3 * (1 + tau) * z.double().abs()) * R.E
    assert ((out[1].double() - q).abs() <= off * q + 1e-37).all()
    assert ((out[0].double() - a).abs() <= torch.where(q < 0.5, off * q + (3 if tau == 1 else 1) * R.E * a, 2 ** s * off * a) + 1e-37).all()
    unit = (q * (1 + a)).sqrt()  # half the relative error of each factor, a root of 2 e and two products
    assert ((out[2].double() - unit).abs() <= (2 ** s * off + 4 * R.E) * unit + 1e-18).all()


def test_not_a_number_stays_in_its_channel_and_after_its_token(L):
    t = make(2, 200, 1, 32, seed=13)
    t["x"][1, 100, 0, 3] = float("nan")
    y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"])
    bad = torch.isnan(y)
    assert bad[1, 100:, 0, 3].all() and bad.sum() == 100 and torch.isnan(h).sum() == 1


def test_the_same_call_gives_the_same_bits(L):
    t = make(3, 900, 2, 64, dtype="bf16", seed=14)
    one, two = both(L, t), both(L, t)
    assert all(torch.equal(one[k], two[k]) for k in one)


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 2, 16), (5, 1, 37), (256, 32, 128)], ids=str)
@pytest.mark.parametrize("dtype,zdtype,head", [("f32", "f32", False), ("bf16", "bf16", False), ("f16", "f32", True)])
def test_step(L, shape, dtype, zdtype, head):
    B, H, d = shape
    if head and d not in (16, 32, 64, 128):
        pytest.skip("a gate per head has the library's head widths")
    for gate, write, tau in (("logit", "leaky", 1.0), ("logit", "unit", 0.25), ("value", "plain", 1.0)):
        t = make(B, 1, H, d, dtype=dtype, zdtype=zdtype, gate=gate, head=head, seed=15)
        ref = R.scan(t["x"], t["z"], t["h0"], gate, write, tau)
        x, z, h = t["x"][:, 0], t["z"][:, 0], t["h0"].clone()
        out = torch.empty_like(h)
        y = L.gated_step(h, x, z, gate=gate, write=write, tau=tau, h_out=out)
        assert torch.equal(h, t["h0"])
        y2 = L.gated_step(h, x, z, gate=gate, write=write, tau=tau)  # in place
        assert torch.equal(h, out) and torch.equal(y, y2)
        R.check(out.unsqueeze(1), {"y": ref["y"], "b_y": ref["b_y"]}, "y")
        R.check(y.unsqueeze(1), ref, "y")
        ys, hs = L.gated_scan_fwd(t["x"], t["z"], t["h0"], gate=gate, write=write, tau=tau)
        assert torch.equal(hs, out) and torch.equal(ys[:, 0], y)  # one token through the scan


def test_offsets_beyond_32_bits(L):
    """One sequence whose rows reach past 2^31 elements."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 20 GB")
    T, wide = 300, 8_000_000  # element offset of the last row: 2.4e9
    buf = torch.empty((1, T, wide), dtype=torch.bfloat16, device="cuda")
    t = make(1, T, 1, 64, dtype="bf16", seed=16)
    want = both(L, t)
    for k, name in enumerate(("x", "z", "dy")):
        v = buf[:, :, k * 64:(k + 1) * 64].unflatten(-1, (1, 64))
        v.copy_(t[name])
        t[name] = v
    got = both(L, t)
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_streams_and_graphs(L):
    t = make(2, 300, 2, 64, dtype="bf16", seed=17)
    want = both(L, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    marks = L.gated_scan_marks(t["x"])
    y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"], marks=marks, stream=side)
    g = L.gated_scan_bwd(t["x"], t["z"], t["dy"], marks, dh_T=t["dh_T"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want["y"]) and torch.equal(g["dz"], want["dz"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m2 = L.gated_scan_marks(t["x"])
        y2, h2 = L.gated_scan_fwd(t["x"], t["z"], t["h0"], marks=m2)
        g2 = L.gated_scan_bwd(t["x"], t["z"], t["dy"], m2, dh_T=t["dh_T"])
    t2 = make(2, 300, 2, 64, dtype="bf16", seed=18)
    for k in ("x", "z", "h0", "dy", "dh_T"):
        t[k].copy_(t2[k])
    graph.replay()
    want = both(L, t2)
    got = {"y": y2, "h_T": h2, **g2}
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("workload", ["small_train", "mid_layer"])
def test_full_sizes_on_sampled_channels(L, workload):
    """The repository's training shapes; every channel is its own recurrence, so the 64-bit
    form runs on a sample of them."""
    import lattice_inputs as LI
    w = LI.WORKLOADS[workload]
    t = make(w.B, w.T, w.H, w.d, dtype="bf16", seed=19, mean=3.0)
    kw = dict(write="unit")
    marks = L.gated_scan_marks(t["x"])
    y, h = L.gated_scan_fwd(t["x"], t["z"], t["h0"], marks=marks, **kw)
    got = L.gated_scan_bwd(t["x"], t["z"], t["dy"], marks, dh_T=t["dh_T"], **kw)
    got.update(y=y, h_T=h)
    pick = (slice(w.B - 1, w.B), slice(None), slice(w.H - 1, w.H), slice(w.d - 8, w.d))
    pick_h = (pick[0], pick[2], pick[3])
    c = {k: t[k][pick if t[k].dim() == 4 else pick_h].contiguous() for k in ("x", "z", "h0", "dy", "dh_T")}
    ref = R.scan(c["x"], c["z"], c["h0"], "logit", "unit", 1.0, None, c["dy"], c["dh_T"])
    for name in ("y", "h_T", "dx", "dz", "dh0"):
        R.check(got[name][pick if got[name].dim() == 4 else pick_h], ref, name)
