"""Which kernels a call launches, from the nodes of a graph that it is captured into."""
import ctypes as C

import torch


class _Dim3(C.Structure):
    _fields_ = [(n, C.c_uint32) for n in "xyz"]


class _Params(C.Structure):
    _fields_ = [("block", _Dim3), ("extra", C.c_void_p), ("func", C.c_void_p), ("grid", _Dim3),
                ("params", C.c_void_p), ("shared", C.c_uint32)]


def launches(call):
    """(name, grid) of each kernel that `call` launches, in order.  The names are the mangled
    ones; nothing is run."""
    hip = C.CDLL("libamdhip64.so.7")
    hip.hipKernelNameRefByPtr.restype = C.c_char_p
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = C.c_void_p(graph.raw_cuda_graph()), C.c_size_t()
    assert hip.hipGraphGetNodes(raw, None, C.byref(n)) == 0
    nodes = (C.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(raw, nodes, C.byref(n)) == 0
    got = []
    for node in nodes:
        kind, p = C.c_int(), _Params()
        assert hip.hipGraphNodeGetType(C.c_void_p(node), C.byref(kind)) == 0
        if kind.value != 0:  # (not a kernel)
            continue
        assert hip.hipGraphKernelNodeGetParams(C.c_void_p(node), C.byref(p)) == 0
        name = hip.hipKernelNameRefByPtr(C.c_void_p(p.func), None)
        got.append((name.decode(), (p.grid.x, p.grid.y, p.grid.z)))
    return got
