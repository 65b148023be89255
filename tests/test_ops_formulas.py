"""The 64-bit forms that the GPU tests compare with: their gradients against central
differences of their forward passes, on the CPU."""
import itertools

import pytest
import torch

import gated_ref
import norm_ref

H = 1e-5


def test_bench_byte_models():
    import bench
    import lattice_inputs as LI
    w = LI.WORKLOADS["mid_layer"]  # 8 * 4096 * 16 * 128 elements, 16 * 128 channels of 8 sequences
    assert bench.gated_alg_bytes(w, False) == 67108864 * 6 + 8 * 2048 * 4
    assert bench.gated_alg_bytes(w, True) == 67108864 * 10 + 8 * 2048 * 4


def differences(loss, t):
    out = torch.zeros_like(t)
    flat, grad = t.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + H
        up = loss()
        flat[i] = keep - H
        down = loss()
        flat[i] = keep
        grad[i] = (up - down) / (2 * H)
    return out


@pytest.mark.parametrize("gate,write,tau,head", [(g, w, t, h) for g, w, t, h in itertools.product(
    ("value", "logit"), ("plain", "leaky", "unit"), (1.0, 0.3), (False, True)) if g == "logit" or t == 1.0])
def test_gated_recurrence(gate, write, tau, head):
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, T, Hh, d = 2, 5, 2, 3
    x, z, h0 = n(B, T, Hh, d), n(B, T, Hh) if head else n(B, T, Hh, d), n(B, Hh, d)
    if gate == "value":
        z = torch.tanh(z) * 0.9
    dy, dh = n(B, T, Hh, d), n(B, Hh, d)
    lens = [5, 3]

    def loss():
        o = gated_ref.scan(x, z, h0, gate, write, tau, lens)
        return ((o["y"] * dy).sum() + (o["h_T"] * dh).sum()).item()
    got = gated_ref.scan(x, z, h0, gate, write, tau, lens, dy, dh)
    for t, name in ((x, "dx"), (z, "dz"), (h0, "dh0")):
        assert torch.allclose(got[name], differences(loss, t), rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("act", ["gelu", "silu", "sigmoid", None])
@pytest.mark.parametrize("post,pre,residual", list(itertools.product((True, False), repeat=3)))
def test_block_norms(act, post, pre, residual):
    gen = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    N, D = 3, 5
    y, g, res = n(N, D), n(N, D) if act else None, n(N, D) if residual else None
    wq, wp, dr, dn = 1 + 0.3 * n(D), 1 + 0.3 * n(D), n(N, D), n(N, D)

    def loss():
        o, _ = norm_ref.forward(y, wq, g, act, res, wp, pre, post, -0.7, 1e-3)
        return ((o["r"] * dr).sum() + ((o["n"] * dn).sum() if pre else 0)).item()
    got = norm_ref.backward(y, wq, g, act, res, wp, post, -0.7, 1e-3, dr, dn if pre else None)
    for t, name in ((y, "dy"), (g, "dgate"), (res, "dresidual"), (wq, "dw_post"), (wp if pre else None, "dw_pre")):
        if t is not None:
            assert torch.allclose(got[name], differences(loss, t), rtol=1e-6, atol=1e-7), name
