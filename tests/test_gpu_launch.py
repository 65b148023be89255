"""How the layer operators' launches stand beside each other in one process: a kernel's grid,
and its results, do not depend on which other calls were made before or are made at once."""
import ctypes
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    import orthogonal_update_recurrent_b200 as L
    from orthogonal_update_recurrent_b200 import build
    build.build()
    return L


class _KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p)] + [(f, ctypes.c_uint) for f in ("gx", "gy", "gz", "bx", "by", "bz", "shared")] \
        + [("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def grids(f):
    """(CTAs, threads) of every kernel that f launches, read from its capture."""
    driver = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        f()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert driver.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert driver.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(-1), _KernelNode()
        assert driver.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert driver.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append((p.gx, p.bx))
    return out


def norm_grids(before):
    """Grids of the norms' forward passes whose CTAs have 256 threads, in a process of its own,
    with or without a backward pass of as many threads before them."""
    import orthogonal_update_recurrent_b200 as L
    wide = torch.randn(8192, 2048, device="cuda").bfloat16()
    heads = torch.randn(65536, 128, device="cuda").bfloat16()
    torch.cuda.synchronize()
    out = []
    for y in (wide, heads):
        if before:
            L.block_norm_bwd(y[:512], residual=y[:512], dr=y[:512], dn=y[:512])
        out += grids(lambda: L.block_norm_fwd(y, residual=y, pre_norm=True))
    return out


def test_a_norm_kernels_grid_is_its_own(L):
    """A forward pass gets the CTAs that the device holds of its kernel, not of one that ran
    before it: these hold twice as many as the backward pass's."""
    got = [subprocess.run([sys.executable, "-c", f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]\n"
                           f"import test_gpu_launch as t\nprint(t.norm_grids({before}))"],
                          check=True, capture_output=True, text=True, timeout=300).stdout for before in (False, True)]
    assert got[0] == got[1]
    assert got[0].count("(") == 2
