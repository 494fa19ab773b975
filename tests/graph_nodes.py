"""Launch shapes of captured calls, read from the graph's nodes."""
from __future__ import annotations

import ctypes

import torch


class _KernelParams(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS (v2) of the driver's interface."""
    _fields_ = ([("func", ctypes.c_void_p)]
                + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "smem")]
                + [(n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")])


def captured_grids(call):
    """CTAs of each kernel that `call` launches on the current stream (which must not allocate)."""
    cu = ctypes.CDLL("libcuda.so.1")
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t()
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(), _KernelParams()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append(p.gx * p.gy * p.gz)
    return out
