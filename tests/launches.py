"""How many kernels a call launches: the nodes of a graph that it is captured into, by the driver's interface."""
import ctypes

import torch


def launches(call):
    """Nodes that call(stream) leaves in a graph; nothing runs."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert cu.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), 2) == 0        # relaxed: other threads' calls are free
    try:
        call(stream)
    finally:
        status = cu.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph))
    assert status == 0 and cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    assert cu.cuGraphDestroy(graph) == 0
    return n.value
