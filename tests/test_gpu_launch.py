"""How the layer operators' launches stand beside each other in one process: a kernel's grid,
and its results, do not depend on which other calls were made before or are made at once."""
import ctypes
import os
import subprocess
import sys
import threading
import time

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


def recorded(L, f):
    """The library call that f makes, as (function, arguments), and what f returned."""
    library, calls = L.lib(), []

    class Recorder:
        def __getattr__(self, name):
            fn = getattr(library, name)

            def call(*args):
                calls.append((fn, args))
                return fn(*args)
            return call if name.startswith("lattice_") and not name.endswith("bytes") else fn
    L.lib, real = lambda: Recorder(), L.lib
    try:
        out = f()
    finally:
        L.lib = real
    assert len(calls) == 1
    return calls[0], out


def at_once(L, fs, seconds=2.0):
    """Repeats the library calls of fs, each on a host thread of its own, and counts those that fail."""
    calls = [recorded(L, f) for f in fs]
    torch.cuda.synchronize()
    failed, start = [0] * len(fs), threading.Barrier(len(fs))

    def repeat(k):
        fn, args = calls[k][0]
        start.wait()
        end = time.monotonic() + seconds
        while time.monotonic() < end:
            for _ in range(100):
                failed[k] += fn(*args) != 0
    switch = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=repeat, args=(k,)) for k in range(len(fs))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(switch)
    torch.cuda.synchronize()
    return failed


def normal(*shape, dtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("head", [False, True])
def test_gated_calls_of_two_host_threads(L, dtype, head):
    """Shapes of one kernel that take clusters of different sizes, and so of different shared memory."""
    sets = []
    for B, T, H in ((1, 5000, 1), (64, 2, 16), (1, 900, 1)):
        x, dy = normal(B, T, H, 64, dtype=dtype), normal(B, T, H, 64, dtype=dtype, seed=1)
        z = normal(B, T, H, dtype=dtype) if head else normal(B, T, H, 64, dtype=dtype, seed=2)
        marks = L.gated_scan_marks(x)
        y, h = L.gated_scan_fwd(x, z, marks=marks)
        sets.append((x, z, dy, marks, y, h, L.gated_scan_bwd(x, z, dy, marks)))
    assert at_once(L, [lambda s=s: L.gated_scan_fwd(s[0], s[1], y=s[4], h_out=s[5]) for s in sets]) == [0, 0, 0]
    assert at_once(L, [lambda s=s: L.gated_scan_bwd(*s[:4]) for s in sets]) == [0, 0, 0]
    for x, z, dy, marks, y, h, g in sets:
        again, state = L.gated_scan_fwd(x, z)
        assert torch.equal(again, y) and torch.equal(state, h)
        grads = L.gated_scan_bwd(x, z, dy, marks)
        assert all(torch.equal(grads[k], g[k]) for k in g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_calls_of_two_host_threads(L, dtype):
    """Widths of one kernel that take different shared memory."""
    for back, widths in ((False, (8192, 6000)), (True, (4096, 2888)), (True, (8192, 6000))):
        sets = []
        for D in widths:
            y, w = normal(8, D, dtype=dtype), normal(D, seed=1)
            out = L.block_norm_fwd(y, w)[0]
            sets.append((y, out, L.block_norm_bwd(y, dr=y)["dy"], w))
        if back:
            assert at_once(L, [lambda s=s: L.block_norm_bwd(s[0], dr=s[0]) for s in sets]) == [0, 0]
        else:
            assert at_once(L, [lambda s=s: L.block_norm_fwd(s[0], s[3], r_out=s[1]) for s in sets]) == [0, 0]
        for y, out, dy, w in sets:
            assert torch.equal(L.block_norm_fwd(y, w)[0], out) and torch.equal(L.block_norm_bwd(y, dr=y)["dy"], dy)


@pytest.mark.parametrize("B,H,ms,chunk", [(200, 1, (16, 64), 1), (200, 1, (16, 64), 8), (200, 1, (68, 128), 1), (1, 2, (40, 100), 1),
                                          (1, 2, (40, 100), 16)])
@pytest.mark.parametrize("mode", ["sim", "dec"])
def test_state_recurrence_calls_of_two_host_threads(L, B, H, ms, chunk, mode):
    """Slot counts of one kernel, on one CTA per sequence and in clusters: CUDA-core scan, and the
    token-by-token backward pass."""
    T, d, sets = 16, 64, []
    for m in ms:
        ins = (normal(B, T, H, d), torch.sigmoid(normal(B, T, H, m, seed=1)), normal(B, T, H, m, seed=2),
               torch.sigmoid(normal(B, T, H, seed=3)), torch.nn.functional.normalize(normal(B, H, m, d, seed=4), dim=-1))
        kw = dict(chunk=chunk, mode=mode)
        sets.append((ins, kw, L.scan_fwd(*ins, **kw)))
    assert at_once(L, [lambda s=s: L.scan_fwd(*s[0], **s[1]) for s in sets], 1.0) == [0, 0]
    if mode == "sim" and chunk == 1:
        dy = normal(B, T, H, d, seed=5)
        room = [torch.empty(L.scan_bwd_workspace_bytes(B, T, H, m, d), dtype=torch.uint8, device="cuda") for m in ms]
        assert at_once(L, [lambda s=s, w=w: L.scan_bwd(*s[0], dy, workspace=w) for s, w in zip(sets, room)], 1.0) == [0, 0]
    for ins, kw, (y, S) in sets:
        again, state = L.scan_fwd(*ins, **kw)
        assert torch.equal(again, y) and torch.equal(state, S)


def status_times():
    """Microseconds of a status check before any layer operator's call, and after calls of all
    types and directions, in a process of its own."""
    import orthogonal_update_recurrent_b200 as L

    def each(n=200):
        best = float("inf")
        for _ in range(5):
            start = time.perf_counter()
            for _ in range(n):
                L.device_status()
            best = min(best, (time.perf_counter() - start) / n)
        return best * 1e6
    x = normal(1, 40, 1, 16)
    torch.cuda.synchronize()
    L.device_status()
    before = each()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        v = x.to(dtype)
        marks = L.gated_scan_marks(v)
        L.gated_scan_fwd(v, v, marks=marks)
        L.gated_scan_bwd(v, v, v, marks)
        L.block_norm_fwd(v)
        L.block_norm_bwd(v, dr=v)
    return before, each()


def test_a_status_check_reads_what_can_have_failed(L):
    """Units of the layer operators that nothing was launched of are not read: there are 6 other
    units, and 9 of these, at about 12 us each."""
    code = (f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]\n"
            "import test_gpu_launch as t\nprint(*t.status_times())")
    out = subprocess.run([sys.executable, "-c", code], check=True, capture_output=True, text=True, timeout=300).stdout
    before, after = map(float, out.split())
    assert before < 0.7 * after, (before, after)


def calls_after_a_failed_one():
    """A status check inside a capture is refused by CUDA. What the next calls return."""
    import orthogonal_update_recurrent_b200 as L
    h, x = torch.zeros(2, 2, 64, device="cuda"), torch.ones(2, 2, 64, device="cuda")
    S = torch.ones(2, 2, 16, 64, device="cuda")
    q = torch.ones(2, 2, 16, device="cuda")
    out = [L.gated_step(h, x, x), L.readout(S, q)]
    torch.cuda.synchronize()
    for f in (lambda: L.gated_step(h.zero_(), x, x), lambda: L.readout(S, q)):
        code = 0
        try:
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                try:
                    L.device_status()
                except L.LatticeError as e:
                    code = e.code
        except RuntimeError:  # the capture was given up
            pass
        assert code == L.ERR_CUDA
        assert torch.equal(f(), out.pop(0))


def test_an_error_is_reported_once(L):
    code = (f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]\n"
            "import test_gpu_launch as t\nt.calls_after_a_failed_one()")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.parametrize("mode", ["sim", "dec"])
def test_decode_calls_of_two_host_threads(L, mode):
    """Slot counts of one kernel, as many heads as make the decode step persistent."""
    sets = []
    for m in (8, 16, 32):
        S, x, c, q, mu = (normal(200, 1, m, 64), normal(200, 1, 64), torch.sigmoid(normal(200, 1, m)), normal(200, 1, m),
                          torch.sigmoid(normal(200, 1)))
        sets.append((torch.nn.functional.normalize(S, dim=-1), x, c, q, mu))
    assert at_once(L, [lambda s=s: L.step(*s, mode=mode) for s in sets], 1.0) == [0, 0, 0]
    for S, x, c, q, mu in sets:
        assert torch.isfinite(S).all()
