"""The launches of a call: it is captured into a graph, which is read and never
run.  Test infrastructure only."""
import ctypes

import torch

from free_ffn_activation_amd import prox as P

_THREAD_LOCAL = 1  # hipStreamCaptureModeThreadLocal
_KERNEL = 0        # hipGraphNodeTypeKernel


class _Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class _KernelNode(ctypes.Structure):
    _fields_ = [("block", _Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", _Dim3),
                ("args", ctypes.c_void_p), ("shared", ctypes.c_uint32)]


def launches(call):
    """[(kernel's mangled name, blocks, threads of a block)] of call(stream)."""
    hip = P.raw_library()  # the HIP runtime's functions are found through it
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p

    def ok(status):
        assert status == 0, f"HIP error {status}"
    stream = torch.cuda.Stream()
    handle = ctypes.c_void_p(stream.cuda_stream)
    torch.cuda.synchronize()
    graph = ctypes.c_void_p()
    ok(hip.hipStreamBeginCapture(handle, _THREAD_LOCAL))
    try:
        call(stream)
    finally:
        end = hip.hipStreamEndCapture(handle, ctypes.byref(graph))
    ok(end)
    try:
        count = ctypes.c_size_t(0)
        ok(hip.hipGraphGetNodes(graph, None, ctypes.byref(count)))
        nodes = (ctypes.c_void_p * count.value)()
        ok(hip.hipGraphGetNodes(graph, nodes, ctypes.byref(count)))
        found = []
        for node in nodes:
            kind, p = ctypes.c_int(-1), _KernelNode()
            ok(hip.hipGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
            assert kind.value == _KERNEL, f"a node of type {kind.value}"
            ok(hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)))
            name = hip.hipKernelNameRefByPtr(ctypes.c_void_p(p.func), None)
            found.append((name.decode() if name else "", p.grid.x * p.grid.y * p.grid.z, p.block.x * p.block.y * p.block.z))
        return found
    finally:
        ok(hip.hipGraphDestroy(graph))
