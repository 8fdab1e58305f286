"""Which kernels a call launches, from a capture of it that never runs."""
import ctypes

import torch


class _Node(ctypes.Structure):
    # the driver's parameters of a kernel node
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def threads_of(call):
    """The threads of a block of each kernel that ``call()`` launches, in ascending order."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    cu, graph, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes, out = (ctypes.c_void_p * n.value)(), []
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        kind, p = ctypes.c_int(-1), _Node()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:  # a kernel
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append(p.block[0] * p.block[1] * p.block[2])
    return sorted(out)
