"""Which form of the product kernel a call takes: the host's rules, restated, and the launch itself as a graph records it.

"cluster": the blocks of a cluster share a tile's K (few tiles); "pairs": two blocks a tile of 256 rows; "one": a block a tile."""
import ctypes

import torch

SPLITS = ((8, 4, 66), (6, 8, 66), (5, 8, 66), (4, 2, 100), (3, 2, 80), (2, 2, 100))   # blocks, blocks of K each, % of the SMs


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def form_of(rows, groups, N, K, expected=0):
    """rows: what the arrays hold, or expected: what a group is said to hold."""
    tiles = min((rows + groups * 127) // 128, rows) * -(-N // 256)
    for split, blocks, percent in SPLITS:
        if K // 128 >= split * blocks and tiles * split * 100 <= sms() * percent:
            return "cluster"
    per = expected or rows // groups
    return "pairs" if -(-per // 128) * 4 >= -(-per // 256) * 7 else "one"


def tiles_of(counts, N, form):
    """(tiles of the groups, blocks or pairs that share them)."""
    rows, units = (256, sms() // 2) if form == "pairs" else (128, sms())
    return sum(-(-c // rows) for c in counts) * -(-N // 256), units


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """[(kernel name, blocks)] of call(stream), recorded on a stream of its own and not run; call allocates nothing."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph, n = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t()
    torch.cuda.synchronize()

    def ok(code):
        assert code == 0, f"driver status {code}"
    ok(cu.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), 2))        # relaxed
    try:
        call(stream)
    finally:
        ok(cu.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph)))
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (ctypes.c_void_p * n.value)()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    got = []
    for node in nodes:
        p, name = KernelNode(), ctypes.c_char_p()
        ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
        if p.func:
            ok(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
        else:
            ok(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)))
        got.append((name.value.decode(), p.grid[0]))
    ok(cu.cuGraphDestroy(graph))
    return got


def form_launched(call):
    """The form of the one product kernel that call(stream) launches."""
    (name, _), = launches(call)
    assert "gemm_kernel" in name, name
    forms = {"Li1ELb0E": "one", "Li2ELb0E": "pairs", "Li1ELb1E": "cluster"}
    return next(form for mark, form in forms.items() if mark in name)
