"""Which kernels a call launches: the call is captured into a graph, which runs
nothing, and the graph's kernel nodes are asked for their names."""

import ctypes
import re

import torch


class _Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint), ("y", ctypes.c_uint), ("z", ctypes.c_uint)]


class _KernelNode(ctypes.Structure):
    _fields_ = [("block", _Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", _Dim3),
                ("params", ctypes.c_void_p), ("lds", ctypes.c_uint)]


def _runtime():
    """The HIP runtime that this process has loaded."""
    with open("/proc/self/maps") as f:
        path = next(line.split()[-1] for line in f if "libamdhip64" in line)
    hip = ctypes.CDLL(path)
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    hip.hipKernelNameRefByPtr.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    hip.hipGraphGetNodes.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]
    hip.hipGraphKernelNodeGetParams.argtypes = [ctypes.c_void_p, ctypes.POINTER(_KernelNode)]
    return hip


def kernel_names(call):
    """The (mangled) names of the kernels that `call` launches on the current stream."""
    call()                                  # what a first call sets up is not captured
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    hip, raw, n = _runtime(), graph.raw_cuda_graph(), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    names = []
    for node in nodes:
        k = _KernelNode()
        assert hip.hipGraphKernelNodeGetParams(node, ctypes.byref(k)) == 0
        names.append(hip.hipKernelNameRefByPtr(k.func, None).decode())
    return names


def tiles(call):
    """The contraction kernels of a call: ("tiled", AS, MS, WHOLE) or
    ("direct", CF, MS, LINES, SPLIT), in order."""
    found = []
    for name in kernel_names(call):
        m = re.search(r"k_(tiled|direct)I(.*?)EEv", name)
        if m:
            found.append((m.group(1),) + tuple(int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2) + "E")))
    return found
