"""Which kernels a call launches: it is captured on a stream of its own, and the graph's kernel nodes are
asked for their names and sizes (the driver's own functions; nothing runs)."""
import ctypes
import re

import torch

_drv = None


class _Node(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS of the driver API, version 2."""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _driver():
    global _drv
    if _drv is None:
        _drv = ctypes.CDLL("libcuda.so.1")
    return _drv


def _ok(name, *args):
    status = getattr(_driver(), name)(*args)
    assert status == 0, (name, status)


def launched(call):
    """[(mangled name, CTAs)] of the kernels that call(stream) launches, in stream order.  The call has to
    have run before, so that what it looks up the first time is there."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph, n = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t(0)
    _ok("cuStreamBeginCapture_v2", handle, 2)                      # relaxed
    try:
        call(side)
    finally:
        _ok("cuStreamEndCapture", handle, ctypes.byref(graph))
    _ok("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    _ok("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    out = []
    for node in nodes:
        kind, p, name = ctypes.c_int(), _Node(), ctypes.c_char_p()
        _ok("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:                                         # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        _ok("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(p))
        if p.func:
            _ok("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(p.func))
        else:
            _ok("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(p.kern))
        out.append((name.value.decode(), p.grid[0] * p.grid[1] * p.grid[2]))
    _ok("cuGraphDestroy", graph)
    return out


def form(call):
    """The gated kernel that a call launches: 'decode', 'stream', 'stream shared' or 'pair', 'pair shared'
    ('shared': several CTAs or pairs have a tile's K), and the CTAs of its grid."""
    for name, ctas in launched(call):
        if "gated_decode_kernel" in name:
            return "decode", ctas
        m = re.search(r"gated_stream(_block)?_kernelILi\d+ELi\d+ELb([01])E", name)
        if m:
            return ("stream shared" if m[2] == "1" else "stream"), ctas
        m = re.search(r"gemm_kernelILi\d+ELi\d+ELi\d+ELb([01])E", name)
        if m:
            return ("pair shared" if m[1] == "1" else "pair"), ctas
    raise AssertionError("no gated kernel was launched")
