"""ctypes binding of libmoe.so: argument marshalling only.

Function names follow include/moe.h.  Device buffers are torch tensors on the
current HIP device; the stream is torch's current stream.  Nothing here
computes any part of the layer: every step runs in the library.  If the
library is missing the import fails loudly -- there is no fallback path.
"""

import ctypes
import functools
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_ESHAPE, MOE_EFORMAT, MOE_EWORKSPACE, MOE_EDEVICE, MOE_ECODE, MOE_ETIMEOUT = \
    0, -1, -2, -3, -4, -5, -6, -7
MOE_ACT_MXFP8 = 1
FMT = {"TERN160": 1, "Q2_0": 2, "Q3": 3, "MXFP4": 4, "Q8": 5}
FMT_NAME = {v: k for k, v in FMT.items()}
MAX_DECODE_ROWS = 8
MAX_TOP_K = 8
MAX_GROUPS = 1024
MAX_Q4_ROWS = 64
T_F32, T_BF16, T_F16 = 0, 1, 2

# every symbol include/moe.h declares
EXPORTS = ("moe_status_string", "moe_packed_bytes", "moe_pack", "moe_unpack",
           "moe_workspace_bytes", "moe_check_experts", "moe_route", "moe_expert_ffn",
           "moe_layer", "moe_layer_profiled", "moe_stack_decode", "moe_quant_mxfp8",
           "moe_stream_read", "moe_set_spin_limit", "moe_workspace_status", "moe_layer_noalloc",
           "moe_allocate_formats", "moe_cache_create", "moe_cache_destroy", "moe_cache_plan",
           "moe_copy_share", "moe_cpu_expert_ffn", "moe_add_chain",
           "moe_group_plan_bytes", "moe_group_plan", "moe_group_matmul", "moe_group_swiglu",
           "moe_group_matmul_t", "moe_group_swiglu_grad", "moe_group_wgrad", "moe_group_combine",
           "moe_group_combine_grad", "moe_q4_bytes", "moe_q4_pack", "moe_q4_unpack", "moe_q4_matvec")


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {status} ({status_string(status)})")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("sel_bias", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("experts", ctypes.c_void_p),
                ("shared", ctypes.c_void_p)]


class ExpertRef(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("gate", ctypes.c_uint64), ("up", ctypes.c_uint64), ("down", ctypes.c_uint64)]


class GroupDims(ctypes.Structure):
    _fields_ = [("n_groups", ctypes.c_int32), ("rows", ctypes.c_int32), ("x_rows", ctypes.c_int32),
                ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("src_div", ctypes.c_int32),
                ("type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("ldx", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("ldw", ctypes.c_int64), ("w_stride", ctypes.c_int64),
                ("ld_pre", ctypes.c_int64)]


class CombineDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n", ctypes.c_int32),
                ("o_rows", ctypes.c_int32), ("type", ctypes.c_int32), ("out_type", ctypes.c_int32),
                ("ldo", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class Q4Dims(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("group", ctypes.c_int32),
                ("n_mats", ctypes.c_int32), ("rows", ctypes.c_int32), ("x_div", ctypes.c_int32),
                ("type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("swiglu", ctypes.c_int32),
                ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


EXPERT_REF_DTYPE = np.dtype([("fmt", "<u4"), ("reserved", "<u4"), ("gate", "<u8"),
                             ("up", "<u8"), ("down", "<u8")])
assert EXPERT_REF_DTYPE.itemsize == ctypes.sizeof(ExpertRef) == 32

_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m bit_moe_expert_02_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        dims_p = ctypes.POINTER(Dims)
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_packed_bytes.restype = sz
        L.moe_packed_bytes.argtypes = [ctypes.c_int, i64, i64]
        L.moe_pack.restype = ctypes.c_int
        L.moe_pack.argtypes = [ctypes.c_int, vp, i64, i64, vp, sz, ctypes.c_int]
        L.moe_unpack.restype = ctypes.c_int
        L.moe_unpack.argtypes = [ctypes.c_int, vp, sz, i64, i64, vp, ctypes.c_int]
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [dims_p, i32]
        L.moe_check_experts.restype = ctypes.c_int
        L.moe_check_experts.argtypes = [dims_p, vp, i32, sz]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [dims_p, vp, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_expert_ffn.restype = ctypes.c_int
        L.moe_expert_ffn.argtypes = [dims_p, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_layer.restype = ctypes.c_int
        L.moe_layer.argtypes = [dims_p, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_layer_noalloc.restype = ctypes.c_int
        L.moe_layer_noalloc.argtypes = [dims_p, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_layer_profiled.restype = ctypes.c_int
        L.moe_layer_profiled.argtypes = [dims_p, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                         vp, vp, i32]
        L.moe_quant_mxfp8.restype = ctypes.c_int
        L.moe_quant_mxfp8.argtypes = [vp, i32, i32, vp, vp, vp]
        L.moe_set_spin_limit.restype = ctypes.c_int32
        L.moe_set_spin_limit.argtypes = [i32]
        L.moe_stream_read.restype = ctypes.c_int
        L.moe_stream_read.argtypes = [vp, sz, vp, i32, i32, vp]
        L.moe_workspace_status.restype = ctypes.c_int
        L.moe_workspace_status.argtypes = [vp, sz, vp]
        L.moe_allocate_formats.restype = ctypes.c_int
        L.moe_allocate_formats.argtypes = [i32, i32, vp, vp, vp, vp, ctypes.c_double, i32, i32, i32, vp,
                                           vp, vp]
        L.moe_stack_decode.restype = ctypes.c_int
        L.moe_stack_decode.argtypes = [dims_p, i32, ctypes.POINTER(LayerWeights), i32, vp, vp, vp,
                                       vp, vp, vp, sz, vp]
        L.moe_cache_create.restype = ctypes.c_int
        L.moe_cache_create.argtypes = [i32, i32, i32, ctypes.POINTER(vp)]
        L.moe_cache_destroy.restype = None
        L.moe_cache_destroy.argtypes = [vp]
        L.moe_cache_plan.restype = ctypes.c_int
        L.moe_cache_plan.argtypes = [vp, i32, i32, i32, vp, ctypes.c_double, vp, vp, vp, vp, vp, vp, vp]
        L.moe_copy_share.restype = ctypes.c_double
        L.moe_copy_share.argtypes = [ctypes.c_double, ctypes.c_double]
        L.moe_cpu_expert_ffn.restype = ctypes.c_int
        L.moe_cpu_expert_ffn.argtypes = [dims_p, i32, vp, vp, vp, vp, i32, vp, vp, vp, i32]
        L.moe_add_chain.restype = ctypes.c_int
        L.moe_add_chain.argtypes = [vp, vp, vp, vp, i32, i32, vp]
        gd_p, cd_p, qd_p = (ctypes.POINTER(c) for c in (GroupDims, CombineDims, Q4Dims))
        sz_p = ctypes.POINTER(sz)
        L.moe_group_plan_bytes.restype = sz
        L.moe_group_plan_bytes.argtypes = [i32, i32, i32]
        for name, args in (("moe_group_plan", [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]),
                           ("moe_group_matmul", [gd_p, vp, vp, vp, vp, vp, vp]),
                           ("moe_group_swiglu", [gd_p, vp, vp, vp, vp, vp, vp, vp]),
                           ("moe_group_matmul_t", [gd_p, vp, vp, vp, vp, vp, vp]),
                           ("moe_group_swiglu_grad", [gd_p, vp, vp, vp, vp, vp, vp, vp]),
                           ("moe_group_wgrad", [gd_p, vp, vp, vp, vp, vp, i32, vp]),
                           ("moe_group_combine", [cd_p, vp, vp, vp, vp, vp]),
                           ("moe_group_combine_grad", [cd_p, vp, vp, vp, vp, vp, vp, vp]),
                           ("moe_q4_bytes", [i64, i64, i32, sz_p, sz_p, sz_p]),
                           ("moe_q4_pack", [vp, i64, i64, i32, vp, vp, vp, i32]),
                           ("moe_q4_unpack", [vp, vp, vp, i64, i64, i32, vp, i32]),
                           ("moe_q4_matvec", [qd_p, vp, vp, vp, vp, vp, vp, vp])):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = args
        _lib = L
    return _lib


def status_string(status):
    return lib().moe_status_string(int(status)).decode()


def _check(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st)


# ----------------------------------------------------------------------------- host packer
def packed_bytes(fmt, n, k):
    return int(lib().moe_packed_bytes(FMT[fmt], int(n), int(k)))


def pack(fmt, w, nthreads=0):
    """fp32 [n, k] (numpy) -> packed uint8 array (numpy), via moe_pack."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    nbytes = packed_bytes(fmt, n, k)
    if nbytes == 0:
        raise MoeError("moe_packed_bytes", MOE_ESHAPE)
    out = np.empty(nbytes, np.uint8)
    _check("moe_pack", lib().moe_pack(FMT[fmt], w.ctypes.data, n, k, out.ctypes.data, nbytes,
                                      int(nthreads)))
    return out


def pack_into(fmt, w, out, nthreads=0):
    """Packs into a preallocated uint8 numpy array view (for large buffers)."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    _check("moe_pack", lib().moe_pack(FMT[fmt], w.ctypes.data, n, k, out.ctypes.data, out.size,
                                      int(nthreads)))


def unpack(fmt, buf, n, k, nthreads=0):
    buf = np.ascontiguousarray(buf, dtype=np.uint8)
    out = np.empty((n, k), np.float32)
    _check("moe_unpack", lib().moe_unpack(FMT[fmt], buf.ctypes.data, buf.size, int(n), int(k),
                                          out.ctypes.data, int(nthreads)))
    return out


def allocate_formats(err, tokens, energy, fmt_bytes, max_tern_frac=0.5, min_tokens=8, edge_first=2,
                     edge_last=3):
    """moe_allocate_formats: err [L, E, 3] (TERN160, Q2_0, Q3), tokens [L, E],
    energy [L], fmt_bytes [3] -> (format names [L, E], total cost, total bytes)."""
    err = np.ascontiguousarray(err, np.float64)
    tokens = np.ascontiguousarray(tokens, np.int32)
    energy = np.ascontiguousarray(energy, np.float64)
    fb = np.ascontiguousarray(fmt_bytes, np.uint64)
    L_, E_ = tokens.shape
    out = np.empty((L_, E_), np.uint8)
    cost = ctypes.c_double()
    nbytes = ctypes.c_uint64()
    _check("moe_allocate_formats", lib().moe_allocate_formats(
        L_, E_, err.ctypes.data, tokens.ctypes.data, energy.ctypes.data, fb.ctypes.data,
        float(max_tern_frac), int(min_tokens), int(edge_first), int(edge_last), out.ctypes.data,
        ctypes.byref(cost), ctypes.byref(nbytes)))
    names = np.vectorize(FMT_NAME.get)(out)
    return names, cost.value, int(nbytes.value)


# ----------------------------------------------------------------------------- device calls
def dims(hidden, inter, n_experts, top_k, flags=0):
    return Dims(hidden, inter, n_experts, top_k, flags)


def workspace_bytes(d, rows):
    return int(lib().moe_workspace_bytes(ctypes.byref(d), int(rows)))


def check_experts(d, table, weights_bytes):
    table = np.ascontiguousarray(table, dtype=EXPERT_REF_DTYPE)
    return int(lib().moe_check_experts(ctypes.byref(d), table.ctypes.data, len(table),
                                       int(weights_bytes)))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # the handle alone: 0.1 us instead of 3
    if raw is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(raw(torch.cuda.current_device()))


def moe_route(d, x, rows, w_router, bias, idx, wts, ws, stream=None):
    _check("moe_route", lib().moe_route(ctypes.byref(d), _ptr(x), int(rows), _ptr(w_router),
                                        _ptr(bias), _ptr(idx), _ptr(wts), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_ffn(d, x, rows, idx, wts, weights, experts, shared, y, ws, stream=None):
    _check("moe_expert_ffn", lib().moe_expert_ffn(
        ctypes.byref(d), _ptr(x), int(rows), _ptr(idx), _ptr(wts), _ptr(weights), _ptr(experts),
        _ptr(shared), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_layer(d, x, rows, w_router, bias, weights, experts, shared, idx, wts, y, ws, stream=None):
    _check("moe_layer", lib().moe_layer(
        ctypes.byref(d), _ptr(x), int(rows), _ptr(w_router), _ptr(bias), _ptr(weights),
        _ptr(experts), _ptr(shared), _ptr(idx), _ptr(wts), _ptr(y), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_layer_noalloc(d, x, rows, w_router, bias, weights, experts, shared, idx, wts, y, stream=None):
    """moe_layer on the library's fixed per-GPU workspace (no allocation)."""
    _check("moe_layer_noalloc", lib().moe_layer_noalloc(
        ctypes.byref(d), _ptr(x), int(rows), _ptr(w_router), _ptr(bias), _ptr(weights),
        _ptr(experts), _ptr(shared), _ptr(idx), _ptr(wts), _ptr(y), _stream(stream)))


def moe_layer_profiled(d, x, rows, w_router, bias, weights, experts, shared, idx, wts, y, ws,
                       events, stream=None):
    arr = (ctypes.c_void_p * len(events))(*events)
    _check("moe_layer_profiled", lib().moe_layer_profiled(
        ctypes.byref(d), _ptr(x), int(rows), _ptr(w_router), _ptr(bias), _ptr(weights),
        _ptr(experts), _ptr(shared), _ptr(idx), _ptr(wts), _ptr(y), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream), arr, len(events)))


def layer_weights(layers):
    """ctypes array of LayerWeights for objects with router, bias, weights, experts, shared."""
    arr = (LayerWeights * len(layers))()
    for i, dl in enumerate(layers):
        addr = [None if t is None else t.data_ptr()
                for t in (dl.router, dl.bias, dl.weights, dl.experts, dl.shared)]
        arr[i] = LayerWeights(*addr)
    return arr


def moe_stack_decode(d, layers, rows, x_all, noise, y_all, idx_all, wts_all, ws, stream=None):
    """layers: a LayerWeights array (layer_weights()); the other buffers are torch tensors."""
    _check("moe_stack_decode", lib().moe_stack_decode(
        ctypes.byref(d), len(layers), layers, int(rows), _ptr(x_all), _ptr(noise), _ptr(y_all),
        _ptr(idx_all), _ptr(wts_all), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_quant_mxfp8(x, rows, k, codes, scales, stream=None):
    _check("moe_quant_mxfp8", lib().moe_quant_mxfp8(_ptr(x), int(rows), int(k), _ptr(codes),
                                                    _ptr(scales), _stream(stream)))


def moe_stream_read(buf, nbytes, sink, grid, unroll, stream=None):
    """Measurement aid: the streaming-read kernel over the first nbytes of buf."""
    _check("moe_stream_read", lib().moe_stream_read(_ptr(buf), int(nbytes), _ptr(sink), int(grid),
                                                    int(unroll), _stream(stream)))


def moe_workspace_status(ws, stream=None):
    """MOE_OK or MOE_ETIMEOUT (a fused call's hand-off wait gave up since the
    last query); synchronises the stream and clears the workspace's error word."""
    st = lib().moe_workspace_status(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    if st not in (MOE_OK, MOE_ETIMEOUT):
        raise MoeError("moe_workspace_status", st)
    return st


def moe_set_spin_limit(polls):
    """Polls before a hand-off wait of the fused launch gives up; returns the previous limit."""
    prev = lib().moe_set_spin_limit(int(polls))
    if prev < 0:
        raise MoeError("moe_set_spin_limit", prev)
    return prev


# ----------------------------------------------------------------------------- stacks larger than HBM
class SlotCache:
    """moe_cache_create / moe_cache_plan / moe_cache_destroy (host only)."""

    def __init__(self, n_layers, n_experts, n_slots):
        h = ctypes.c_void_p()
        _check("moe_cache_create", lib().moe_cache_create(int(n_layers), int(n_experts), int(n_slots),
                                                          ctypes.byref(h)))
        self.h, self.n_experts, self.n_slots = h, int(n_experts), int(n_slots)

    def plan(self, layer, idx, copy_share):
        """idx: host int32 [rows, top_k] -> dict(slot_of [E], copies [(expert, slot)],
        cpu [experts], idx_gpu [rows, top_k])."""
        idx = np.ascontiguousarray(idx, np.int32)
        rows, k = idx.shape
        n = rows * k
        slot_of = np.empty(self.n_experts, np.int32)
        ce, cs, cpu, idx_gpu = (np.empty(max(n, 1), np.int32) for _ in range(4))
        nc, nu = ctypes.c_int32(), ctypes.c_int32()
        _check("moe_cache_plan", lib().moe_cache_plan(
            self.h, int(layer), rows, k, idx.ctypes.data, float(copy_share), slot_of.ctypes.data,
            ce.ctypes.data, cs.ctypes.data, ctypes.byref(nc), cpu.ctypes.data, ctypes.byref(nu),
            idx_gpu.ctypes.data))
        return {"slot_of": slot_of,
                "copies": [(int(ce[i]), int(cs[i])) for i in range(nc.value)],
                "cpu": [int(cpu[i]) for i in range(nu.value)],
                "idx_gpu": idx_gpu[:n].reshape(rows, k).copy()}

    def close(self):
        if self.h:
            lib().moe_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def copy_share(pcie_bytes_per_s, cpu_bytes_per_s):
    return float(lib().moe_copy_share(float(pcie_bytes_per_s), float(cpu_bytes_per_s)))


def cpu_expert_ffn(d, fmt, gate, up, down, x_bf16, row_ids, row_w, y, nthreads=0):
    """moe_cpu_expert_ffn on host numpy arrays: y [rows, H] fp32 accumulates
    row_w[j] * FFN(x[row_ids[j]])."""
    for a in (gate, up, down, x_bf16, y):
        assert a.flags.c_contiguous
    assert y.dtype == np.float32
    rid = np.ascontiguousarray(row_ids, np.int32)
    rw = np.ascontiguousarray(row_w, np.float32)
    _check("moe_cpu_expert_ffn", lib().moe_cpu_expert_ffn(
        ctypes.byref(d), FMT[fmt] if isinstance(fmt, str) else int(fmt), gate.ctypes.data,
        up.ctypes.data, down.ctypes.data, x_bf16.ctypes.data, len(rid), rid.ctypes.data,
        rw.ctypes.data, y.ctypes.data, int(nthreads)))


def moe_add_chain(y, add, noise, x_next, stream=None):
    """y [rows, hidden] fp32 device tensor; add / noise likewise or None; x_next
    [rows, hidden] int16 (bf16 bits) or None."""
    rows, hidden = y.shape
    _check("moe_add_chain", lib().moe_add_chain(_ptr(y), _ptr(add), _ptr(noise), _ptr(x_next),
                                                int(rows), int(hidden), _stream(stream)))


# ----------------------------------------------------------------------------- experts at any shape
# Shapes, strides and types are read off the tensors (torch, on the current
# device, last dimension contiguous); what does not fit raises MoeError.  A
# small call is bound by this module, so each check is made once.
_types = {}


def _type_of(t):
    code = _types.get(t.dtype)
    if code is None and not _types:
        import torch
        _types.update({torch.float32: T_F32, torch.bfloat16: T_BF16, torch.float16: T_F16, torch.int32: -1})
        code = _types.get(t.dtype)
    return -2 if code is None else code


def _type(fn, t):
    code = _type_of(t)
    if code < 0:
        raise MoeError(fn, MOE_EFORMAT)
    return code


def _need(fn, ok, status=MOE_ESHAPE):
    if not ok:
        raise MoeError(fn, status)


_hooks = None


def _device_hooks():
    """(current device, current raw stream of a device): torch's own cheap forms of both where it has them."""
    global _hooks
    import torch
    device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream)
    _hooks = (device, stream)
    return _hooks


def _addresses(fn, stream, *tensors):
    """The stream's handle, then the addresses of tensors (None: None) that have to lie on the current device."""
    dev = tensors[0].get_device()
    if dev < 0:
        raise MoeError(fn, MOE_EINVAL)
    device, current = _hooks or _device_hooks()
    if dev != device():
        raise MoeError(fn, MOE_EINVAL)
    out = [current(dev) if stream is None else stream.cuda_stream]
    for t in tensors:
        if t is None:
            out.append(None)
        else:
            if t.get_device() != dev:
                raise MoeError(fn, MOE_EINVAL)
            out.append(t.data_ptr())
    return out


def _rows(fn, t):
    """(rows, columns, row stride) of a 2-d tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise MoeError(fn, MOE_ESHAPE)
    (r, c), (ld, one) = t.shape, t.stride()
    if one != 1 and c > 1:
        raise MoeError(fn, MOE_ESHAPE)
    return r, c, ld if r > 1 else max(ld, c)


def _ints(fn, t, n):
    if _types.get(t.dtype) != -1 and _type_of(t) != -1:
        raise MoeError(fn, MOE_EFORMAT)
    if t.numel() != n or not t.is_contiguous():
        raise MoeError(fn, MOE_ESHAPE)


def group_plan_bytes(rows, top_k, n_groups):
    return int(lib().moe_group_plan_bytes(int(rows), int(top_k), int(n_groups)))


def moe_group_plan(idx, n_groups, offsets, pairs, pos, ws=None, stream=None):
    """idx [rows, top_k] int32 -> offsets [n_groups + 1], pairs and pos [rows * top_k] (all int32);
    ws: group_plan_bytes(rows, top_k, n_groups) bytes, or None when that is 0."""
    fn = "moe_group_plan"
    st, *at = _addresses(fn, stream, idx, offsets, pairs, pos, ws)
    _need(fn, idx.dim() == 2)
    rows, top_k = idx.shape
    n = rows * top_k
    for t, count in ((idx, n), (offsets, n_groups + 1), (pairs, n), (pos, n)):
        _ints(fn, t, count)
    _need(fn, ws is None or ws.is_contiguous())
    _check(fn, lib().moe_group_plan(at[0], rows, top_k, int(n_groups), at[1], at[2], at[3], at[4],
                                    0 if ws is None else ws.numel() * ws.element_size(), st))


def _group_dims(fn, x, src, src_div, offsets, rows, w, out):
    """(GroupDims with everything but ldy and ld_pre, columns of x), x the operand that src selects rows of."""
    kind, out_type = _types.get(x.dtype, -2), _types.get(out.dtype, -2)
    if kind < 0 or out_type < 0:
        kind, out_type = _type(fn, x), _type(fn, out)
    if w.dim() != 3:
        raise MoeError(fn, MOE_ESHAPE)
    (groups, n, k), (stride, ldw, one) = w.shape, w.stride()
    if groups < 1 or (one != 1 and k > 1):
        raise MoeError(fn, MOE_ESHAPE)
    _ints(fn, offsets, groups + 1)
    if src is not None:
        _ints(fn, src, rows)
    x_rows, x_cols, ldx = _rows(fn, x)
    return GroupDims(groups, rows, x_rows, n, k, src_div, kind, out_type, ldx, 0, ldw if n > 1 else max(k, ldw),
                     stride if groups > 1 else 0, 0), x_cols


def _product(fn, call, x, offsets, w, y, src, src_div, back, stream, pre=None, factor=None):
    """factor: None without pre, else the columns of (y, pre) per column of the product, times two."""
    s, xa, oa, wa, ya, sa, pa = _addresses(fn, stream, x, offsets, w, y, src, pre)
    rows, y_cols, ldy = _rows(fn, y)
    d, x_cols = _group_dims(fn, x, src, src_div, offsets, rows, w, y)
    d.ldy = ldy
    x_want, cols = (d.n, d.k) if back else (d.k, d.n)
    if x.dtype != w.dtype or x_cols != x_want or 2 * y_cols != cols * (factor[0] if factor else 2):
        raise MoeError(fn, MOE_ESHAPE)
    if factor is None:
        st = call(d, xa, sa, oa, wa, ya, s)
    else:
        if pre is not None:
            p_rows, p_cols, d.ld_pre = _rows(fn, pre)
            if pre.dtype != x.dtype or p_rows != rows or 2 * p_cols != cols * factor[1]:
                raise MoeError(fn, MOE_ESHAPE)
        st = call(d, xa, sa, oa, wa, pa, ya, s) if back else call(d, xa, sa, oa, wa, ya, pa, s)
    if st:
        raise MoeError(fn, st)


def moe_group_matmul(x, offsets, w, y, src=None, src_div=1, stream=None):
    """y [rows, n] = x[src // src_div] [., k] times w [groups, n, k] of each row's group, transposed."""
    _product("moe_group_matmul", lib().moe_group_matmul, x, offsets, w, y, src, src_div, False, stream)


def moe_group_swiglu(x, offsets, w, h, pre=None, src=None, src_div=1, stream=None):
    """h [rows, n / 2] = silu(gate) * up of (gate | up) = the product with w [groups, n, k]; pre [rows, n]
    (gate | up) in x's type, or None."""
    _product("moe_group_swiglu", lib().moe_group_swiglu, x, offsets, w, h, src, src_div, False, stream, pre, (1, 2))


def moe_group_matmul_t(dy, offsets, w, dx, src=None, src_div=1, stream=None):
    """dx [rows, k] = dy [., n] times w [groups, n, k] of each row's group."""
    _product("moe_group_matmul_t", lib().moe_group_matmul_t, dy, offsets, w, dx, src, src_div, True, stream)


def moe_group_swiglu_grad(dy, offsets, w, pre, dpre, src=None, src_div=1, stream=None):
    """dpre [rows, 2 k]: the gradient of (gate | up) = pre [rows, 2 k] from dy [., n], the gradient of the
    product of h = silu(gate) * up with w [groups, n, k]."""
    _need("moe_group_swiglu_grad", pre is not None, MOE_EINVAL)
    _product("moe_group_swiglu_grad", lib().moe_group_swiglu_grad, dy, offsets, w, dpre, src, src_div, True, stream, pre,
             (4, 4))


def moe_group_wgrad(dy, x, offsets, dw, src=None, src_div=1, accumulate=False, stream=None):
    """dw [groups, n, k] = (or +=) dy[rows of the group]^T x[src // src_div of those rows]."""
    fn = "moe_group_wgrad"
    s, dya, xa, oa, dwa, sa = _addresses(fn, stream, dy, x, offsets, dw, src)
    rows, n, ldy = _rows(fn, dy)
    d, x_cols = _group_dims(fn, x, src, src_div, offsets, rows, dw, dw)
    d.ldy = ldy
    if dy.dtype != x.dtype or x_cols != d.k or n != d.n:
        raise MoeError(fn, MOE_ESHAPE)
    _check(fn, lib().moe_group_wgrad(d, dya, xa, sa, oa, dwa, 1 if accumulate else 0, s))


def _combine_dims(fn, o_rows, ldo, y, pos, wts, top_k, in_type, out_type):
    rows, n, ldy = _rows(fn, y)
    if pos is not None:
        _ints(fn, pos, rows * top_k)
    if wts is not None and (_type(fn, wts) != T_F32 or wts.shape != (rows, top_k) or not wts.is_contiguous()):
        raise MoeError(fn, MOE_ESHAPE)
    return CombineDims(rows, top_k, n, o_rows, in_type, out_type, ldo, ldy)


def _top_k(fn, rows, pos, wts, o_rows, top_k):
    if top_k is None:
        top_k = wts.shape[-1] if wts is not None else (pos.numel() if pos is not None else o_rows) // max(rows, 1)
    return int(top_k)


def moe_group_combine(o, pos, wts, y, top_k=None, stream=None):
    """y [rows, n] = sum over a row's top_k pairs of wts * o[pos]; pos None: pair p is row p; wts None: 1."""
    fn = "moe_group_combine"
    s, oa, pa, wa, ya = _addresses(fn, stream, o, pos, wts, y)
    kind, out = _type(fn, o), _type(fn, y)
    o_rows, n, ldo = _rows(fn, o)
    d = _combine_dims(fn, o_rows, ldo, y, pos, wts, _top_k(fn, y.shape[0], pos, wts, o_rows, top_k), kind, out)
    _need(fn, d.n == n)
    _check(fn, lib().moe_group_combine(d, oa, pa, wa, ya, s))


def moe_group_combine_grad(dy, o, pos, wts, d_o, d_wts, top_k=None, stream=None):
    """d_o[pos] = wts * dy (rows of d_o that no pair names stay as they were) and d_wts = <dy, o[pos]>; either
    output may be None.  o (None without d_wts) and d_o have the same row stride."""
    fn = "moe_group_combine_grad"
    s, dya, oa, pa, wa, doa, dwa = _addresses(fn, stream, dy, o, pos, wts, d_o, d_wts)
    like = d_o if d_o is not None else o
    _need(fn, like is not None and (d_wts is None or o is not None), MOE_EINVAL)
    kind, out = _type(fn, dy), _type(fn, like)
    o_rows, n, ldo = _rows(fn, like)
    if o is not None:
        _need(fn, o.dtype == dy.dtype and _rows(fn, o) == (o_rows, n, ldo))
    top_k = _top_k(fn, dy.shape[0], pos, wts, o_rows, top_k if d_wts is None else d_wts.shape[-1])
    d = _combine_dims(fn, o_rows, ldo, dy, pos, wts, top_k, kind, out)
    _need(fn, d.n == n)
    if d_wts is not None:
        _need(fn, _type(fn, d_wts) == T_F32 and d_wts.is_contiguous() and d_wts.shape == (d.rows, top_k))
    _check(fn, lib().moe_group_combine_grad(d, dya, oa, pa, wa, doa, dwa, s))


# ----------------------------------------------------------------------------- 4-bit matrix-vector products
def q4_bytes(n, k, group):
    """(codes, scales, zeros) bytes of a packed n x k matrix."""
    out = [ctypes.c_size_t() for _ in range(3)]
    _check("moe_q4_bytes", lib().moe_q4_bytes(int(n), int(k), int(group), *(ctypes.byref(v) for v in out)))
    return tuple(int(v.value) for v in out)


def q4_pack(w, group, zeros=False, nthreads=0):
    """fp32 [n, k] (numpy) -> (codes uint8, scales uint8, zeros uint8 or None) (numpy), via moe_q4_pack."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    nc, ns, nz = q4_bytes(n, k, group)
    codes, scales, zr = np.empty(nc, np.uint8), np.empty(ns, np.uint8), np.empty(nz, np.uint8) if zeros else None
    _check("moe_q4_pack", lib().moe_q4_pack(w.ctypes.data, n, k, int(group), codes.ctypes.data, scales.ctypes.data,
                                            None if zr is None else zr.ctypes.data, int(nthreads)))
    return codes, scales, zr


def q4_unpack(codes, scales, zeros, n, k, group, nthreads=0):
    bufs = [None if b is None else np.ascontiguousarray(b).view(np.uint8).reshape(-1) for b in (codes, scales, zeros)]
    for b, need in zip(bufs, q4_bytes(n, k, group)):
        _need("moe_q4_unpack", b is None or b.size >= need)
    out = np.empty((n, k), np.float32)
    _check("moe_q4_unpack", lib().moe_q4_unpack(*(None if b is None else b.ctypes.data for b in bufs), int(n), int(k),
                                                int(group), out.ctypes.data, int(nthreads)))
    return out


def moe_q4_matvec(x, codes, scales, zeros, group, y, idx=None, x_div=1, swiglu=False, n_mats=None, stream=None):
    """y[p] = W x[p // x_div] for the rows p of y, W the matrix idx.flatten()[p] (idx None: matrix 0); swiglu:
    W = (gate | up), y = silu(gate) * up.  codes / scales / zeros (or None): the packed matrices back to back;
    n_mats defaults to the first dimension of codes when it has more than one, else 1."""
    fn = "moe_q4_matvec"
    s, xa, ca, sa, za, ya, ia = _addresses(fn, stream, x, codes, scales, zeros, y, idx)
    kind, out = _type(fn, x), _type(fn, y)
    x_rows, k, ldx = _rows(fn, x)
    rows, n, ldy = _rows(fn, y)
    if swiglu:
        n *= 2
    if n_mats is None:
        n_mats = codes.shape[0] if codes.dim() > 1 else 1
    if idx is not None:
        _ints(fn, idx, rows)
    _need(fn, x_div >= 1 and (rows == 0 or x_rows > (rows - 1) // x_div))
    for t, need in zip((codes, scales, zeros), _q4_sizes(n, k, group)):
        if t is not None and (t.numel() * t.element_size() < need * n_mats or not t.is_contiguous()):
            raise MoeError(fn, MOE_ESHAPE)
    d = Q4Dims(n, k, group, n_mats, rows, x_div, kind, out, 1 if swiglu else 0, ldx, ldy)
    _check(fn, lib().moe_q4_matvec(d, xa, ia, ca, sa, za, ya, s))


@functools.lru_cache(maxsize=256)
def _q4_sizes(n, k, group):
    return q4_bytes(n, k, group)
