"""What the gated recurrence and the block norms refuse, on the host: every call below fails
its checks before any CUDA call (none could run here), through the C ABI and the binding."""
import ctypes

import pytest
import torch

import orthogonal_update_recurrent_b200 as L
from orthogonal_update_recurrent_b200 import build as B

M = 1 << 20
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def p(a):
    return None if a is None else ctypes.c_void_p(a)


def scan(lib, **kw):
    a = dict(x=1 * M, xd=BF16, xb=4 * 64, xt=64, z=2 * M, zd=BF16, zb=4 * 64, zt=64, head=0, h0=3 * M, ho=4 * M, y=5 * M, marks=None,
             lens=None, B=2, T=4, H=2, d=32, gate=1, write=1, tau=1.0)
    a.update(kw)
    return lib.lattice_gated_scan_fwd(p(a["x"]), a["xd"], a["xb"], a["xt"], p(a["z"]), a["zd"], a["zb"], a["zt"], a["head"],
                                      p(a["h0"]), p(a["ho"]), p(a["y"]), p(a["marks"]), p(a["lens"]), a["B"], a["T"], a["H"],
                                      a["d"], a["gate"], a["write"], a["tau"], None)


INVALID = L.ERR_INVALID_ARG
UNSUPPORTED = L.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(z=None), INVALID), (dict(y=None), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(xd=3), INVALID), (dict(zd=-1), INVALID), (dict(gate=2), INVALID),
    (dict(write=3), INVALID), (dict(write=-1), INVALID), (dict(tau=0.0), INVALID), (dict(tau=-1.0), INVALID),
    (dict(tau=float("nan")), INVALID), (dict(tau=float("inf")), INVALID), (dict(xb=-1), INVALID), (dict(zt=-64), INVALID),
    (dict(x=M + 1), INVALID), (dict(zd=F32, z=2 * M + 2), INVALID), (dict(h0=3 * M + 2), INVALID), (dict(marks=6 * M + 8), INVALID),
    (dict(lens=7 * M + 1), INVALID),
    (dict(y=1 * M + 64), INVALID), (dict(ho=2 * M), INVALID), (dict(ho=3 * M + 16), INVALID), (dict(marks=5 * M), INVALID),
    (dict(y=3 * M + 128), INVALID), (dict(lens=5 * M + 8), INVALID), (dict(xt=1 << 61, T=1 << 10), INVALID),
    (dict(zd=F16), UNSUPPORTED), (dict(xd=F32, zd=BF16), UNSUPPORTED), (dict(head=1, d=24), UNSUPPORTED),
    (dict(head=1, d=256), UNSUPPORTED), (dict(H=1 << 16, d=1 << 15), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
])
def test_scan_forward(lib, kw, code):
    assert scan(lib, **kw) == code


def test_scan_backward(lib):
    def bwd(**kw):
        a = dict(x=1 * M, xd=BF16, z=2 * M, zd=BF16, head=0, dy=3 * M, marks=4 * M, dh=5 * M, dx=6 * M, dz=7 * M, dh0=8 * M, lens=None,
                 B=2, T=40, H=2, d=32, gate=1, write=1, tau=1.0, bs=40 * 64, ts=64)
        a.update(kw)
        return lib.lattice_gated_scan_bwd(p(a["x"]), a["xd"], a["bs"], a["ts"], p(a["z"]), a["zd"], a["bs"], a["ts"], a["head"],
                                          p(a["dy"]), a["bs"], a["ts"], p(a["marks"]), p(a["dh"]), p(a["dx"]), p(a["dz"]),
                                          p(a["dh0"]), p(a["lens"]), a["B"], a["T"], a["H"], a["d"], a["gate"], a["write"],
                                          a["tau"], None)
    for kw in (dict(x=None), dict(dy=None), dict(marks=None), dict(dx=None), dict(dz=None), dict(dh0=None), dict(dx=3 * M + 2),
               dict(dz=6 * M), dict(dh0=5 * M), dict(dx=4 * M), dict(marks=4 * M + 4), dict(ts=-1), dict(tau=0.0)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(zd=F16) == UNSUPPORTED
    # a state before every 16th token
    assert lib.lattice_gated_scan_marks_bytes(2, 40, 2, 32) == 2 * 3 * 64 * 4
    assert lib.lattice_gated_scan_marks_bytes(2, 0, 2, 32) == 0
    assert lib.lattice_gated_scan_marks_bytes(0, 40, 2, 32) == 0


def test_step(lib):
    def step(**kw):
        a = dict(h=1 * M, ho=1 * M, x=2 * M, xd=BF16, z=3 * M, zd=BF16, head=0, y=4 * M, B=2, H=2, d=32, gate=1, write=1, tau=1.0)
        a.update(kw)
        return lib.lattice_gated_step(p(a["h"]), p(a["ho"]), p(a["x"]), a["xd"], 64, p(a["z"]), a["zd"], 64, a["head"], p(a["y"]),
                                      a["B"], a["H"], a["d"], a["gate"], a["write"], a["tau"], None)
    for kw in (dict(h=None), dict(ho=None), dict(x=None), dict(z=None), dict(y=None), dict(ho=1 * M + 16), dict(y=1 * M),
               dict(y=2 * M), dict(ho=3 * M), dict(B=0), dict(gate=5), dict(tau=-2.0)):
        assert step(**kw) == INVALID, kw
    assert step(head=1, d=20) == UNSUPPORTED


def test_norms(lib):
    def fwd(**kw):
        a = dict(y=1 * M, yd=BF16, ys=64, g=None, gs=0, r=2 * M, rd=F32, rs=64, wq=3 * M, wp=4 * M, wd=F32, ro=5 * M, no=6 * M,
                 dt=BF16, N=8, G=1, D=64, act=3, post=1, scale=1.0, eps=1e-6)
        a.update(kw)
        return lib.lattice_block_norm_fwd(p(a["y"]), a["yd"], a["ys"], p(a["g"]), a["gs"], p(a["r"]), a["rd"], a["rs"], p(a["wq"]),
                                          p(a["wp"]), a["wd"], p(a["ro"]), p(a["no"]), a["dt"], a["N"], a["G"], a["D"], a["act"],
                                          a["post"], a["scale"], a["eps"], None)
    for kw in (dict(y=None), dict(ro=None), dict(no=None), dict(N=-1), dict(G=0), dict(G=3), dict(D=0), dict(ys=-1), dict(dt=9),
               dict(yd=4), dict(act=4), dict(act=-1), dict(act=0, g=7 * M), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(scale=float("nan")), dict(y=M + 1), dict(r=2 * M + 2), dict(ro=1 * M), dict(ro=2 * M + 256), dict(no=5 * M),
               dict(no=3 * M), dict(ro=6 * M)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(D=16385), dict(N=1 << 31), dict(yd=F16), dict(rd=F16), dict(wd=F16), dict(ys=1 << 31), dict(dt=F32, yd=BF16)):
        assert fwd(**kw) == UNSUPPORTED, kw
    assert fwd(N=0) == L.OK  # nothing to do

    def bwd(**kw):
        a = dict(y=1 * M, yd=BF16, g=None, r=2 * M, rd=F32, wq=3 * M, wp=4 * M, wd=F32, dr=5 * M, drd=F32, dn=6 * M, dy=7 * M, dg=None,
                 dres=8 * M, dwq=9 * M, dwp=10 * M, ws=11 * M, wsb=M, dt=BF16, N=8, G=1, D=64, act=3, post=1, scale=1.0, eps=1e-6)
        a.update(kw)
        return lib.lattice_block_norm_bwd(p(a["y"]), a["yd"], 64, p(a["g"]), 64, p(a["r"]), a["rd"], 64, p(a["wq"]), p(a["wp"]),
                                          a["wd"], p(a["dr"]), a["drd"], 64, p(a["dn"]), 64, p(a["dy"]), p(a["dg"]), p(a["dres"]),
                                          p(a["dwq"]), p(a["dwp"]), p(a["ws"]), a["wsb"], a["dt"], a["N"], a["G"], a["D"],
                                          a["act"], a["post"], a["scale"], a["eps"], None)
    need = lib.lattice_block_norm_bwd_workspace_bytes(8, 64)
    assert need > 0 and need % (2 * 64 * 4) == 0
    for kw in (dict(dr=None, dn=None, wp=None, dwp=None), dict(dn=None), dict(dy=None), dict(dres=None), dict(g=12 * M),
               dict(dg=12 * M), dict(ws=None), dict(wsb=need - 1), dict(ws=11 * M + 8), dict(wq=None), dict(wp=None), dict(dy=1 * M),
               dict(dres=5 * M), dict(dwq=10 * M), dict(dwp=11 * M), dict(ws=7 * M), dict(drd=8)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(drd=F16), dict(drd=BF16), dict(D=20000)):
        assert bwd(**kw) == UNSUPPORTED, kw
    assert lib.lattice_block_norm_bwd_workspace_bytes(-1, 64) == 0
    assert lib.lattice_block_norm_bwd_workspace_bytes(8, 16385) == 0


def test_scans_of_states_still_refuse_fp16(lib):
    v = ctypes.c_void_p
    assert lib.lattice_scan_fwd_ex(v(M), F16, v(2 * M), v(3 * M), 0, v(4 * M), None, v(5 * M), v(6 * M), v(7 * M), 1, 4, 1, 64, 64,
                                   64, 0, 0, 0, None) == INVALID


def test_binding_rejects_host_tensors():
    x, h = torch.zeros(1, 2, 1, 16), torch.zeros(1, 1, 16)
    with pytest.raises(TypeError):
        L.gated_scan_fwd(x, x, h)
    with pytest.raises(TypeError):
        L.gated_step(h, h, h)
    with pytest.raises(ValueError):
        L.gated_scan_fwd(x[0], x[0])
    with pytest.raises(TypeError):
        L.block_norm_fwd(x, None)
    with pytest.raises(ValueError):
        L.block_norm_bwd(x)
    with pytest.raises(TypeError):
        L.block_norm_bwd(x, dr=x)
