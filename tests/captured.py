"""Which kernels a call launches, from a capture of it in a CUDA graph."""
import ctypes


class KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """(name, CTAs, dynamic shared memory, CTAs an SM holds) of the kernels that `call` launches."""
    import torch
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu, raw, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes, out = (ctypes.c_void_p * n.value)(), []
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        p, name = KernelNode(), ctypes.c_char_p()
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        func, fit = ctypes.c_void_p(p.func), ctypes.c_int()
        if not p.func:
            assert cu.cuKernelGetFunction(ctypes.byref(func), ctypes.c_void_p(p.kern)) == 0
        assert cu.cuFuncGetName(ctypes.byref(name), func) == 0
        assert cu.cuOccupancyMaxActiveBlocksPerMultiprocessor(ctypes.byref(fit), func, p.block[0] * p.block[1] * p.block[2],
                                                              ctypes.c_size_t(p.shared)) == 0
        out.append((name.value.decode(), p.grid[0], p.shared, fit.value))
    return out
