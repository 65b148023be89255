"""What the short convolution, the selective scan and the layer norm refuse, on the host: every call below fails its checks
before any CUDA call (none could run here), through the C ABI and the binding; and what the host computes for them."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import orthogonal_update_recurrent_b200 as L
from orthogonal_update_recurrent_b200 import build as B

M = 1 << 20
F32, BF16, F16 = 0, 1, 2
INVALID, UNSUPPORTED = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def p(a):
    return None if a is None else ctypes.c_void_p(a)


def conv(lib, **kw):
    a = dict(x=1 * M, xd=BF16, xb=40 * 64, xt=64, w=2 * M, bias=3 * M, wd=F32, s=4 * M, so=5 * M, y=6 * M, lens=None, B=2, T=40, C=64,
             K=4, act=2)
    a.update(kw)
    return lib.lattice_short_conv_fwd(p(a["x"]), a["xd"], a["xb"], a["xt"], p(a["w"]), p(a["bias"]), a["wd"], p(a["s"]), p(a["so"]),
                                      p(a["y"]), p(a["lens"]), a["B"], a["T"], a["C"], a["K"], a["act"], None)


def conv_bwd(lib, **kw):
    a = dict(x=1 * M, xd=BF16, xb=40 * 64, xt=64, w=2 * M, bias=3 * M, wd=F32, s=4 * M, dy=5 * M, yb=40 * 64, yt=64, dso=6 * M, dx=7 * M,
             dw=8 * M, db=9 * M, ds=10 * M, ws=11 * M, wsb=M, lens=None, B=2, T=40, C=64, K=4, act=2)
    a.update(kw)
    return lib.lattice_short_conv_bwd(p(a["x"]), a["xd"], a["xb"], a["xt"], p(a["w"]), p(a["bias"]), a["wd"], p(a["s"]), p(a["dy"]),
                                      a["yb"], a["yt"], p(a["dso"]), p(a["dx"]), p(a["dw"]), p(a["db"]), p(a["ds"]), p(a["ws"]),
                                      a["wsb"], p(a["lens"]), a["B"], a["T"], a["C"], a["K"], a["act"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID),
    (dict(C=0), INVALID), (dict(K=0), INVALID), (dict(xd=3), INVALID), (dict(wd=-1), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(xb=-1), INVALID), (dict(xt=-64), INVALID), (dict(x=M + 1), INVALID), (dict(w=2 * M + 2), INVALID),
    (dict(bias=3 * M + 1), INVALID), (dict(s=4 * M + 1), INVALID), (dict(lens=7 * M + 2), INVALID), (dict(y=M + 64), INVALID),
    (dict(so=1 * M), INVALID), (dict(so=4 * M + 128), INVALID), (dict(y=5 * M), INVALID), (dict(y=2 * M), INVALID),
    (dict(xt=1 << 61, T=1 << 10), INVALID), (dict(act=1), UNSUPPORTED), (dict(act=3), UNSUPPORTED), (dict(wd=F16), UNSUPPORTED),
    (dict(xd=F32, wd=BF16), UNSUPPORTED), (dict(K=9), UNSUPPORTED), (dict(C=(1 << 30) + 1), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
])
def test_convolution_forward(lib, kw, code):
    assert conv(lib, **kw) == code


def test_convolution_backward_and_step(lib):
    need = lib.lattice_short_conv_bwd_workspace_bytes(2, 40, 64, 4)
    assert need >= 2 * 5 * 64 * 4 and need % (2 * 5 * 64 * 4) == 0  # a row of 5 weights per channel, at least one per sequence
    for kw in (dict(x=None), dict(dy=None), dict(dx=None), dict(w=None), dict(bias=None), dict(s=None), dict(ws=None), dict(wsb=need - 1),
               dict(ws=11 * M + 8), dict(dx=1 * M), dict(dx=5 * M), dict(dw=7 * M), dict(db=8 * M), dict(ds=4 * M), dict(ds=6 * M), dict(ws=7 * M),
               dict(yt=-1), dict(dy=5 * M + 1), dict(dw=8 * M + 2), dict(dso=6 * M + 1)):
        assert conv_bwd(lib, **kw) == INVALID, kw
    assert conv_bwd(lib, K=9) == UNSUPPORTED and conv_bwd(lib, act=1) == UNSUPPORTED
    for bad in ((0, 40, 64, 4), (2, -1, 64, 4), (2, 40, 0, 4), (2, 40, 64, 0), (2, 40, 64, 9)):
        assert lib.lattice_short_conv_bwd_workspace_bytes(*bad) == 0

    def step(**kw):
        a = dict(s=1 * M, so=1 * M, x=2 * M, xd=BF16, xb=64, w=3 * M, bias=4 * M, wd=BF16, y=5 * M, B=2, C=64, K=4, act=2)
        a.update(kw)
        return lib.lattice_short_conv_step(p(a["s"]), p(a["so"]), p(a["x"]), a["xd"], a["xb"], p(a["w"]), p(a["bias"]), a["wd"], p(a["y"]),
                                           a["B"], a["C"], a["K"], a["act"], None)
    for kw in (dict(s=None), dict(so=None), dict(x=None), dict(w=None), dict(y=None), dict(so=1 * M + 128), dict(y=1 * M), dict(y=2 * M),
               dict(so=3 * M), dict(B=0), dict(xb=-1), dict(K=0)):
        assert step(**kw) == INVALID, kw
    assert step(K=9) == UNSUPPORTED and step(wd=F16) == UNSUPPORTED


SCAN = dict(x=1 * M, xd=BF16, dt=2 * M, dtd=BF16, A=3 * M, b=4 * M, c=5 * M, skip=6 * M, z=7 * M, bias=8 * M, sp=1, rb=40 * 64, rt=64, vb=40 * 16,
            vt=16, B=2, T=40, E=64, N=16, G=1, lens=None)


def scan_args(a):
    return (p(a["x"]), a["xd"], a["rb"], a["rt"], p(a["dt"]), a["dtd"], a["rb"], a["rt"], p(a["A"]), p(a["b"]), a["vb"], a["vt"], p(a["c"]),
            a["vb"], a["vt"], p(a["skip"]), p(a["z"]), a["rb"], a["rt"], p(a["bias"]), a["sp"])


def scan(lib, **kw):
    a = dict(SCAN, h0=9 * M, ho=10 * M, y=11 * M, marks=12 * M, ws=14 * M, wsb=M)
    a.update(kw)
    return lib.lattice_selective_scan_fwd(*scan_args(a), p(a["h0"]), p(a["ho"]), p(a["y"]), p(a["marks"]), p(a["lens"]), p(a["ws"]),
                                          a["wsb"], a["B"], a["T"], a["E"], a["N"], a["G"], None)


def scan_bwd(lib, **kw):
    a = dict(SCAN, dy=9 * M, marks=10 * M, dh=12 * M, dx=13 * M, ddt=14 * M, dA=15 * M, db=16 * M, dc=17 * M, dskip=18 * M, dz=19 * M,
             dbias=20 * M, dh0=21 * M, ws=22 * M, wsb=M)
    a.update(kw)
    return lib.lattice_selective_scan_bwd(*scan_args(a), p(a["dy"]), a["rb"], a["rt"], p(a["marks"]), p(a["dh"]), p(a["dx"]), p(a["ddt"]),
                                          p(a["dA"]), p(a["db"]), p(a["dc"]), p(a["dskip"]), p(a["dz"]), p(a["dbias"]), p(a["dh0"]),
                                          p(a["lens"]), p(a["ws"]), a["wsb"], a["B"], a["T"], a["E"], a["N"], a["G"], None)


SHARED = [
    (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID), (dict(b=None), INVALID), (dict(c=None), INVALID),
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
    (dict(xd=3), INVALID), (dict(dtd=-1), INVALID), (dict(rb=-1), INVALID), (dict(vt=-16), INVALID), (dict(x=M + 1), INVALID),
    (dict(dtd=F32, dt=2 * M + 2), INVALID), (dict(A=3 * M + 2), INVALID), (dict(skip=6 * M + 1), INVALID), (dict(bias=8 * M + 2), INVALID),
    (dict(b=4 * M + 1), INVALID), (dict(lens=13 * M + 2), INVALID), (dict(vt=1 << 61, T=1 << 10), INVALID), (dict(dtd=F16), UNSUPPORTED),
    (dict(xd=F32, dtd=BF16), UNSUPPORTED), (dict(N=129), UNSUPPORTED), (dict(E=(1 << 30) + 1), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(y=None, marks=None), INVALID), (dict(h0=9 * M + 2), INVALID), (dict(marks=12 * M + 8), INVALID), (dict(y=1 * M), INVALID),
    (dict(y=7 * M + 64), INVALID), (dict(ho=2 * M), INVALID), (dict(ho=9 * M + 16), INVALID), (dict(marks=11 * M), INVALID),
    (dict(y=9 * M), INVALID), (dict(ho=3 * M), INVALID),
])
def test_scan_forward(lib, kw, code):
    assert scan(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(dy=None), INVALID), (dict(marks=None), INVALID), (dict(dx=None), INVALID), (dict(ddt=None), INVALID), (dict(dA=None), INVALID),
    (dict(db=None), INVALID), (dict(dc=None), INVALID), (dict(dz=None), INVALID), (dict(z=None), INVALID), (dict(skip=None), INVALID),
    (dict(bias=None), INVALID), (dict(dh0=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=64), INVALID), (dict(ws=22 * M + 4), INVALID),
    (dict(dx=1 * M), INVALID), (dict(ddt=13 * M), INVALID), (dict(db=16 * M, dc=16 * M + 64), INVALID), (dict(dh0=10 * M), INVALID),
    (dict(dA=3 * M), INVALID), (dict(dz=9 * M), INVALID), (dict(ws=21 * M), INVALID), (dict(marks=10 * M + 4), INVALID), (dict(dx=13 * M + 1), INVALID),
])
def test_scan_backward(lib, kw, code):
    assert scan_bwd(lib, **kw) == code


def test_scan_step_and_sizes(lib):
    def step(**kw):
        a = dict(SCAN, h=9 * M, ho=9 * M, y=10 * M)
        a.update(kw)
        return lib.lattice_selective_step(p(a["h"]), p(a["ho"]), p(a["x"]), a["xd"], a["E"], p(a["dt"]), a["dtd"], a["E"], p(a["A"]),
                                          p(a["b"]), a["N"], p(a["c"]), a["N"], p(a["skip"]), p(a["z"]), a["E"], p(a["bias"]), a["sp"],
                                          p(a["y"]), a["B"], a["E"], a["N"], a["G"], None)
    for kw in (dict(h=None), dict(ho=None), dict(x=None), dict(dt=None), dict(A=None), dict(b=None), dict(c=None), dict(y=None),
               dict(ho=9 * M + 16), dict(y=9 * M), dict(y=1 * M), dict(ho=3 * M), dict(B=0), dict(G=5), dict(h=9 * M + 2)):
        assert step(**kw) == INVALID, kw
    assert step(N=129) == UNSUPPORTED and step(dtd=F16) == UNSUPPORTED

    # a state before every 8th token
    assert lib.lattice_selective_scan_marks_bytes(2, 41, 64, 16) == 2 * 6 * 64 * 16 * 4
    assert lib.lattice_selective_scan_marks_bytes(2, 0, 64, 16) == 0
    for bad in ((0, 40, 64, 16), (2, -1, 64, 16), (2, 40, 64, 129)):
        assert lib.lattice_selective_scan_marks_bytes(*bad) == 0
        assert lib.lattice_selective_scan_workspace_bytes(*bad, 1, 1) == 0
    assert lib.lattice_selective_scan_workspace_bytes(2, 40, 64, 16, 5, 1) == 0  # 64 channels are no 5 groups
    # a forward pass that fills the device needs none, a long one of few channels a state per segment and channel at least
    assert lib.lattice_selective_scan_workspace_bytes(64, 4096, 2048, 16, 1, 0) == 0
    assert lib.lattice_selective_scan_workspace_bytes(1, 65536, 1024, 16, 1, 0) >= 2 * 1024 * 16 * 4
    # the backward pass's sums of db and dc over channel tiles
    assert lib.lattice_selective_scan_workspace_bytes(64, 4096, 2048, 16, 1, 1) >= 64 * 4096 * 2 * 16 * 4


def test_layer_norm(lib):
    def fwd(**kw):
        a = dict(x=1 * M, xd=BF16, xs=64, r=2 * M, rd=F32, rs=64, w=3 * M, b=4 * M, wd=F32, ro=5 * M, no=6 * M, dt=BF16, N=8, G=1, D=64, eps=1e-5)
        a.update(kw)
        return lib.lattice_layer_norm_fwd(p(a["x"]), a["xd"], a["xs"], p(a["r"]), a["rd"], a["rs"], p(a["w"]), p(a["b"]), a["wd"], p(a["ro"]),
                                          p(a["no"]), a["dt"], a["N"], a["G"], a["D"], a["eps"], None)
    for kw in (dict(x=None), dict(no=None), dict(ro=None), dict(r=None), dict(N=-1), dict(G=0), dict(G=3), dict(D=0), dict(xs=-1), dict(rs=-1),
               dict(dt=9), dict(xd=4), dict(rd=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(x=M + 1), dict(r=2 * M + 2),
               dict(w=3 * M + 2), dict(ro=1 * M), dict(ro=2 * M + 256), dict(no=5 * M), dict(no=3 * M), dict(no=4 * M)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(D=16385), dict(N=1 << 31), dict(xd=F16), dict(rd=F16), dict(wd=F16), dict(xs=1 << 31), dict(dt=F32)):
        assert fwd(**kw) == UNSUPPORTED, kw
    assert fwd(N=0) == L.OK and fwd(N=0, r=None, ro=None) == L.OK  # nothing to do

    def bwd(**kw):
        a = dict(r=1 * M, rd=F32, dn=2 * M, dr=3 * M, w=4 * M, wd=F32, dro=5 * M, dx=6 * M, xd=BF16, dw=7 * M, db=8 * M, ws=9 * M, wsb=M, dt=BF16,
                 N=8, G=1, D=64, eps=1e-5, s=64)
        a.update(kw)
        return lib.lattice_layer_norm_bwd(p(a["r"]), a["rd"], a["s"], p(a["dn"]), a["s"], p(a["dr"]), a["s"], p(a["w"]), a["wd"], p(a["dro"]),
                                          p(a["dx"]), a["xd"], p(a["dw"]), p(a["db"]), p(a["ws"]), a["wsb"], a["dt"], a["N"], a["G"], a["D"],
                                          a["eps"], None)
    need = lib.lattice_layer_norm_bwd_workspace_bytes(8, 64)
    assert need > 0 and need % (2 * 64 * 4) == 0
    for kw in (dict(r=None), dict(dn=None), dict(dro=None), dict(w=None), dict(ws=None), dict(wsb=need - 1), dict(ws=9 * M + 8), dict(dro=1 * M),
               dict(dx=2 * M), dict(dx=5 * M), dict(dw=8 * M), dict(ws=5 * M), dict(xd=7), dict(s=-1), dict(eps=0.0), dict(dw=7 * M + 2)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(rd=F16), dict(xd=F16), dict(D=20000)):
        assert bwd(**kw) == UNSUPPORTED, kw
    assert lib.lattice_layer_norm_bwd_workspace_bytes(-1, 64) == 0 and lib.lattice_layer_norm_bwd_workspace_bytes(8, 16385) == 0


def test_binding_rejects_host_tensors():
    x, w, h = torch.zeros(1, 2, 16), torch.zeros(16, 4), torch.zeros(1, 16, 16)
    A, b = torch.zeros(16, 16), torch.zeros(1, 2, 16)
    for f in (lambda: L.short_conv_fwd(x, w), lambda: L.short_conv_bwd(x, w, x), lambda: L.short_conv_step(x, x[:, 0], w),
              lambda: L.selective_scan_fwd(x, x, A, b, b), lambda: L.selective_scan_bwd(x, x, A, b, b, x, h),
              lambda: L.selective_step(h, x[:, 0], x[:, 0], A, b[:, 0], b[:, 0]), lambda: L.layer_norm_fwd(x),
              lambda: L.layer_norm_bwd(x, x)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: L.short_conv_fwd(x[0], w), lambda: L.selective_scan_fwd(x[0], x, A, b, b), lambda: L.selective_step(h, x, x, A, b, b)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        L.layer_norm_bwd(x, None)


def test_scan_columns_of_the_largest_call(tmp_path):
    """The columns that the scan's backward pass adds up last, by the rule that its launch and its kernel use, where 2 E is no int."""
    main = tmp_path / "columns.cpp"
    main.write_text('#include <stdio.h>\n#include "args.h"\n'
                    'int main() { using namespace lattice; printf("%d %lld %lld", kSelMaxSize, sel_columns(kSelMaxSize, 2),'
                    ' sel_columns(kSelMaxSize, kSelMaxN)); }\n')
    subprocess.run(["g++", "-std=c++17", "-I", B.CSRC, "-o", str(tmp_path / "columns"), str(main)], check=True)
    out = subprocess.run([str(tmp_path / "columns")], check=True, capture_output=True, text=True).stdout
    E = 1 << 30
    assert [int(v) for v in out.split()] == [E, 4 * E, 130 * E]
    for name in ("selective_launch.cuh", "selective_bwd.cuh"):  # the only rule for them there
        with open(os.path.join(B.CSRC, name)) as f:
            text = f.read()
        assert "sel_columns(" in text and not re.search(r"\b2 \* [Aa]\.E\b(?! \+ (A\.E \+ )?p\.column)", text), name


def test_binding_rejects_sizes_that_are_no_int_beside_an_axis_of_0():
    """No tokens, so no elements, of more sequences than an int counts: cut off, they would be one sequence, and the states of the others
    would come back unwritten."""
    many = (1 << 32) + 1
    x, w, A, b = torch.empty(many, 0, 1), torch.empty(1, 2), torch.empty(1, 1), torch.empty(many, 0, 1)
    for f in (lambda: L.short_conv_fwd(x, w), lambda: L.short_conv_bwd(x, w, x), lambda: L.selective_scan_fwd(x, x, A, b, b),
              lambda: L.selective_scan_bwd(x, x, A, b, b, x, b), lambda: L.gated_scan_fwd(x[..., None], x[..., None])):
        with pytest.raises(L.LatticeError):
            f()
