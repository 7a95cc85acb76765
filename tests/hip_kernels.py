"""Which kernels a call launches, and with which grids: it is captured into a graph, whose nodes are
read through the HIP runtime that the process has loaded (GPU tests only)."""
import ctypes

import torch


class _Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class _KernelNode(ctypes.Structure):  # hipKernelNodeParams
    _fields_ = [("block", _Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", _Dim3),
                ("params", ctypes.c_void_p), ("shared", ctypes.c_uint32)]


def _runtime():
    """The HIP runtime of this process: torch's."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64" in line}
    assert len(paths) == 1, paths
    hip = ctypes.CDLL(paths.pop())
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    return hip


def launches_of(call):
    """Of each kernel that call(stream) launches, in no order: its (mangled)
    name, its grid and its workgroup.  The call is recorded and not run."""
    hip = _runtime()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    raw, graph, n = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()

    def do(name, *args):
        rc = getattr(hip, name)(*args)
        assert rc == 0, f"{name}: {rc}"
    do("hipStreamBeginCapture", raw, 2)  # hipStreamCaptureModeRelaxed
    try:
        call(stream)
    finally:
        do("hipStreamEndCapture", raw, ctypes.byref(graph))
    found = []
    try:
        do("hipGraphGetNodes", graph, None, ctypes.byref(n))
        nodes = (ctypes.c_void_p * n.value)()
        do("hipGraphGetNodes", graph, nodes, ctypes.byref(n))
        for node in nodes:
            p = _KernelNode()
            do("hipGraphKernelNodeGetParams", ctypes.c_void_p(node), ctypes.byref(p))
            name = hip.hipKernelNameRefByPtr(ctypes.c_void_p(p.func), raw)
            assert name, "a kernel without a name"
            found.append((name.decode(), (p.grid.x, p.grid.y, p.grid.z), (p.block.x, p.block.y, p.block.z)))
    finally:
        do("hipGraphDestroy", graph)
    return found


def kernels_of(call):
    return [name for name, _, _ in launches_of(call)]
