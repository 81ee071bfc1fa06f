"""Python binding of ``liblora_gemv.so``, the gfx950 heterogeneous-adapter LoRA delta.

Argument marshalling only: every step runs in the HIP kernels behind the C ABI
declared in ``include/lora_gemv.h``.  PyTorch provides device memory and the
stream (the current torch stream unless one is given).  There is no CPU path:
if the library is not built, importing the binding's functions raises.

The calls follow "m07 -- Multi-Adapter (LoRA) Serving", "6. Deep Dive A:
Batching Heterogeneous Adapters": the batch, an index vector mapping each row
to an adapter slot, and an adapter table read on the device.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

__all__ = [
    "LoraError", "Segments", "segment_bound", "ModuleIO", "MODULES", "TABLE_ENTRY_DTYPE", "lib", "workspace_bytes",
    "build_segments", "shrink", "expand", "apply_layer", "apply_layer_noalloc", "decode_layer",
    "decode_layer_launches", "layer_shrink", "layer_expand", "pack_table", "STATIC_SCRATCH_BYTES",
    "status_string", "MAX_RANK", "host_lib", "LinearIO", "LinearQ4IO", "Q4_GROUP", "MASK_INT8_ITEMS", "module_mask",
    "LinearI8IO", "linear_i8_workspace_bytes", "GroupedIO", "grouped_layer", "grouped_workspace_bytes", "pack_weights",
    "WEIGHT_ENTRY_DTYPE", "I8_MAX_IN", "LinearQ4GIO", "linear_q4g_workspace_bytes", "GatedIO", "GatedQ4GIO", "gated_layer",
    "gated_workspace_bytes", "grouped_layer_q4g", "grouped_gated_layer", "grouped_gated_layer_q4g", "pack_weights_q4g",
    "WEIGHT_Q4G_ENTRY_DTYPE", "Q4_GROUPS", "ACTIVATIONS",
]

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblora_gemv.so")
MAX_RANK = 64
STATIC_SCRATCH_BYTES = 16 << 20  # LORA_STATIC_SCRATCH_BYTES
MODULES = ("q", "k", "v", "o", "gate", "up", "down")

# lora_adapter_entry_t, 32 bytes
TABLE_ENTRY_DTYPE = np.dtype([("A", "<u8"), ("B", "<u8"), ("rank", "<i4"), ("scale", "<f4"), ("format", "<i4"),
                              ("reserved", "<i4")])
# lora_weight_entry_t, 32 bytes
WEIGHT_ENTRY_DTYPE = np.dtype([("W", "<u8"), ("Ws", "<u8"), ("ldw", "<i8"), ("reserved", "<i8")])
assert WEIGHT_ENTRY_DTYPE.itemsize == 32
# lora_weight_q4g_entry_t, 32 bytes
WEIGHT_Q4G_ENTRY_DTYPE = np.dtype([("W", "<u8"), ("Ws", "<u8"), ("ldw", "<i8"), ("lds", "<i8")])
Q4_GROUPS = (32, 64, 128)  # inputs that share a scale in the _q4g calls
ACTIVATIONS = ("silu", "gelu_tanh")  # lora_activation_t, in order
I8_MAX_IN = 131072  # LORA_I8_MAX_IN
FORMAT_BF16, FORMAT_INT8_ROWS = 0, 1  # lora_factor_format_t
assert TABLE_ENTRY_DTYPE.itemsize == 32


class LoraError(RuntimeError):
    pass


class _Seg(ctypes.Structure):
    _fields_ = [("perm", ctypes.c_void_p), ("seg_offsets", ctypes.c_void_p), ("seg_adapter", ctypes.c_void_p),
                ("num_segments", ctypes.c_void_p), ("tile_counts", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("max_segments", ctypes.c_int32)]


class _IO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32)]


class _LinIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("W", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32)]


class _LinQ4IO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("Wq", ctypes.c_void_p), ("ldwq", ctypes.c_int64),
                ("Ws", ctypes.c_void_p), ("lds", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32)]


class _LinI8IO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("Wq", ctypes.c_void_p), ("ldwq", ctypes.c_int64),
                ("Ws", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("d_in", ctypes.c_int32),
                ("d_out", ctypes.c_int32)]


class _GroupedIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("rows_per_x", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _LinQ4GIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("Wq", ctypes.c_void_p), ("ldwq", ctypes.c_int64),
                ("Ws", ctypes.c_void_p), ("lds", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _GatedIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("Wg", ctypes.c_void_p), ("ldwg", ctypes.c_int64),
                ("Wu", ctypes.c_void_p), ("ldwu", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_ff", ctypes.c_int32)]


class _GatedQ4GIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("Wgq", ctypes.c_void_p), ("ldwg", ctypes.c_int64),
                ("Wgs", ctypes.c_void_p), ("ldsg", ctypes.c_int64), ("Wuq", ctypes.c_void_p), ("ldwu", ctypes.c_int64),
                ("Wus", ctypes.c_void_p), ("ldsu", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("d_in", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LoraError(f"{LIB_PATH} is missing: build it with `python -m adapter_gemv_amd.build` "
                            "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        st, i32, i64, u32, vp, sz = (ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                     ctypes.c_void_p, ctypes.c_size_t)
        L.lora_workspace_bytes.restype = sz
        L.lora_workspace_bytes.argtypes = [i32, i32, i32, i64]
        L.lora_status_string.restype = ctypes.c_char_p
        L.lora_status_string.argtypes = [st]
        L.lora_build_segments.restype = st
        L.lora_build_segments.argtypes = [vp, i32, i32, _Seg, vp, sz, vp]
        L.lora_shrink.restype = st
        L.lora_shrink.argtypes = [vp, i64, i32, i32, vp, i32, i32, i32, _Seg, i32, vp, i64, vp, sz, vp]
        L.lora_expand.restype = st
        L.lora_expand.argtypes = [vp, i64, i32, i32, vp, i32, i32, i32, _Seg, i32, vp, i64, vp, sz, vp]
        for name in ("lora_apply_layer", "lora_layer_shrink", "lora_layer_expand"):
            f = getattr(L, name)
            f.restype = st
            f.argtypes = [ctypes.POINTER(_IO), u32, i32, vp, i32, _Seg, i32, vp, sz, vp]
        L.lora_decode_layer.restype = st
        L.lora_decode_layer.argtypes = [ctypes.POINTER(_IO), u32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        L.lora_decode_layer_launches.restype = i32
        L.lora_decode_layer_launches.argtypes = [ctypes.POINTER(_IO), u32, i32, i32, _Seg, i32]
        L.lora_apply_layer_noalloc.restype = st
        L.lora_apply_layer_noalloc.argtypes = [ctypes.POINTER(_IO), u32, i32, vp, i32, _Seg, i32, vp]
        L.lora_apply_layer_stacked.restype = st
        L.lora_apply_layer_stacked.argtypes = [ctypes.POINTER(_IO), u32, i32, vp, i32, vp, vp, i32, _Seg, i32, vp, sz,
                                               vp]
        L.lora_linear_workspace_bytes.restype = sz
        L.lora_linear_workspace_bytes.argtypes = [i32, i32, i32, i64, i32]
        for name in ("lora_linear_layer", "lora_linear_shrink", "lora_linear_expand"):
            f = getattr(L, name)
            f.restype = st
            f.argtypes = [ctypes.POINTER(_LinIO), u32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        for name in ("lora_linear_layer_q4", "lora_linear_shrink_q4", "lora_linear_expand_q4"):
            f = getattr(L, name)
            f.restype = st
            f.argtypes = [ctypes.POINTER(_LinQ4IO), u32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        for name in ("lora_linear_layer_i8", "lora_linear_shrink_i8", "lora_linear_expand_i8"):
            f = getattr(L, name)
            f.restype = st
            f.argtypes = [ctypes.POINTER(_LinI8IO), u32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        L.lora_linear_i8_workspace_bytes.restype = sz
        L.lora_linear_i8_workspace_bytes.argtypes = [i32, i32, i32, i64, i32]
        L.lora_grouped_workspace_bytes.restype = sz
        L.lora_grouped_workspace_bytes.argtypes = [i32, i32, i64, i32]
        L.lora_grouped_layer.restype = st
        L.lora_grouped_layer.argtypes = [ctypes.POINTER(_GroupedIO), u32, i32, vp, i32, _Seg, vp]
        L.lora_grouped_layer_i8.restype = st
        L.lora_grouped_layer_i8.argtypes = [ctypes.POINTER(_GroupedIO), u32, i32, vp, i32, _Seg, vp, sz, vp]
        L.lora_linear_q4g_workspace_bytes.restype = sz
        L.lora_linear_q4g_workspace_bytes.argtypes = [i32, i32, i32, i64, i32]
        L.lora_linear_layer_q4g.restype = st
        L.lora_linear_layer_q4g.argtypes = [ctypes.POINTER(_LinQ4GIO), u32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        L.lora_gated_workspace_bytes.restype = sz
        L.lora_gated_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.lora_gated_layer.restype = st
        L.lora_gated_layer.argtypes = [ctypes.POINTER(_GatedIO), i32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        L.lora_gated_layer_q4g.restype = st
        L.lora_gated_layer_q4g.argtypes = [ctypes.POINTER(_GatedQ4GIO), i32, i32, vp, vp, i32, _Seg, i32, vp, sz, vp]
        L.lora_grouped_layer_q4g.restype = st
        L.lora_grouped_layer_q4g.argtypes = [ctypes.POINTER(_GroupedIO), u32, i32, vp, i32, i32, _Seg, vp]
        L.lora_grouped_gated_layer.restype = st
        L.lora_grouped_gated_layer.argtypes = [ctypes.POINTER(_GroupedIO), i32, i32, vp, i32, _Seg, vp]
        L.lora_grouped_gated_layer_q4g.restype = st
        L.lora_grouped_gated_layer_q4g.argtypes = [ctypes.POINTER(_GroupedIO), i32, i32, vp, i32, i32, _Seg, vp]
        L.lora_form_batch.restype = st
        L.lora_form_batch.argtypes = [vp, i32, vp, ctypes.c_float, i32, i32, i32, i32, vp, vp]
        _lib = L
    return _lib


_host = None


def host_lib() -> ctypes.CDLL:
    """The library of the host-only calls (lora_form_batch, lora_status_string):
    liblora_gemv.so, or with LORA_SANITIZE=1 in the environment their
    AddressSanitizer + UndefinedBehaviorSanitizer build liblora_host_san.so
    (``python -m adapter_gemv_amd.build --sanitize``; the process must have
    the sanitizer runtime preloaded)."""
    global _host
    if _host is None:
        if os.environ.get("LORA_SANITIZE") != "1":
            return lib()
        path = os.path.join(HERE, "liblora_host_san.so")
        if not os.path.exists(path):
            raise LoraError(f"{path} is missing: build it with `python -m adapter_gemv_amd.build --sanitize`")
        L = ctypes.CDLL(path)
        L.lora_status_string.restype = ctypes.c_char_p
        L.lora_status_string.argtypes = [ctypes.c_int]
        L.lora_form_batch.restype = ctypes.c_int
        L.lora_form_batch.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float,
                                      ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_void_p, ctypes.c_void_p]
        _host = L
    return _host


def status_string(code: int) -> str:
    return host_lib().lora_status_string(code).decode()


def _check(code: int, what: str):
    if code != 0:
        raise LoraError(f"{what}: {status_string(code)}")


_raw_stream = None  # torch's lookup of the current stream's handle, without a Stream object around it


def _stream(stream):
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()  # initialises the device
        get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        _raw_stream = ((lambda: get(dev())) if get and dev else (lambda: torch.cuda.current_stream().cuda_stream))
    return _raw_stream()


def _rows(t, dtype, rows, cols, dev, name, field):
    """(address, row stride) of a matrix on device `dev` with unit stride along
    its rows, at least `rows` of them and `cols` wide; the checks of _need, in
    few steps for the ordinary case (a decode call marshals up to 28 tensors)."""
    try:
        (n, c), (ld, unit) = t.size(), t.stride()
        if t.dtype is dtype and t.get_device() == dev and n >= rows and c >= cols and (unit == 1 or c <= 1):
            # a single row's stride has no meaning: torch may give any
            return t.data_ptr(), ld if n > 1 else -(-c // 16) * 16
    except (AttributeError, TypeError, ValueError):
        pass
    _need(t, dtype, f"{name}.{field}", 2)
    if t.get_device() != dev:
        raise ValueError(f"{name}.{field} is on another device than the rest of the call")
    if t.shape[0] < rows:
        raise ValueError(f"{name}.{field}: fewer than {rows} rows")
    raise ValueError(f"{name}.{field}: fewer than {cols} columns")


def _slot_table(t, num_slots, what):
    """The device table of num_slots * 7 entries of 32 bytes, whole and in one piece."""
    if t.numel() * t.element_size() < num_slots * (len(MODULES) * 32) or not t.is_contiguous():
        raise ValueError(f"{what}: not the {num_slots} x {len(MODULES)} contiguous entries of 32 bytes that the call reads")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, dtype, what, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{what} must have {ndim} dims")
    if t.dim() >= 1 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have unit stride in its last dim")


class Segments:
    """Device buffers of lora_segments_t for batches of up to ``num_rows`` rows.

    ``max_segments`` (host, 0 = none) bounds the segments of a build: the
    number of distinct valid adapter ids of the batch, which the host that
    formed the batch knows (see ``segment_bound``).  The calls size their
    work items for it; a build with more segments drops those of the highest
    slots and counts their rows into the status word."""

    def __init__(self, num_rows: int, device="cuda", max_segments: int = 0):
        import torch
        n = max(int(num_rows), 1)
        i32 = dict(dtype=torch.int32, device=device)
        self.num_rows = int(num_rows)
        self.max_segments = int(max_segments)
        self.perm = torch.zeros(n, **i32)
        self.seg_offsets = torch.zeros(n + 1, **i32)
        self.seg_adapter = torch.zeros(n, **i32)
        self.num_segments = torch.zeros(1, **i32)
        self.tile_counts = torch.zeros(2, **i32)
        self.status = torch.zeros(1, **i32)

    def c(self) -> _Seg:
        if self.max_segments < 0:
            raise ValueError("max_segments must be >= 0")
        return _Seg(self.perm.data_ptr(), self.seg_offsets.data_ptr(), self.seg_adapter.data_ptr(),
                    self.num_segments.data_ptr(), self.tile_counts.data_ptr(), self.status.data_ptr(),
                    self.max_segments)

    def host(self):
        """(perm, seg_offsets, seg_adapter, status) copied to the host (synchronises)."""
        ns = int(self.num_segments.item())
        offs = self.seg_offsets[:ns + 1].cpu().numpy()
        return (self.perm[:int(offs[-1])].cpu().numpy(), offs, self.seg_adapter[:ns].cpu().numpy(),
                int(self.status.item()))


def segment_bound(row_adapter, num_slots: int) -> int:
    """Host ids (any int array, one per row; for several adapters per row, a
    [rows, depth] array: the most over the columns) -> the distinct valid
    slots, the tightest ``Segments.max_segments`` for a batch (0 when it has
    none)."""
    import numpy as np
    ids = np.asarray(row_adapter)
    if ids.size == 0:
        return 0
    cols = ids.reshape(ids.shape[0], -1).T if ids.ndim > 1 else ids[None]
    return max((int(np.unique(c[(c >= 0) & (c < num_slots)]).size) for c in cols), default=0)


class ModuleIO:
    """One projection for the layer calls: x [rows, >= d_in], y [rows, >= d_out], bf16."""

    def __init__(self, x, y, d_in=None, d_out=None):
        self.x, self.y = x, y
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_out = int(y.shape[1] if d_out is None else d_out)


def workspace_bytes(num_rows: int, num_slots: int, max_rank: int, sum_d_in: int) -> int:
    return int(lib().lora_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in))


class LinearIO:
    """One projection for linear_layer: x [rows, >= d_in], W [d_out, >= d_in]
    (the base weight), y [rows, >= d_out] (written), bf16."""

    def __init__(self, x, W, y, d_in=None, d_out=None):
        self.x, self.W, self.y = x, W, y
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_out = int(W.shape[0] if d_out is None else d_out)


Q4_GROUP = 128  # LORA_Q4_GROUP


class LinearQ4IO:
    """One projection for linear_layer_q4: x [rows, >= d_in] bf16, Wq uint8
    [d_out, >= d_in / 2] (packed signed 4-bit weights, the even input in the
    low nibble), Ws float32 [d_out, >= d_in / Q4_GROUP] (group scales), y
    [rows, >= d_out] bf16 (written).  LinearQ4GIO with group 128 takes the same
    weight and is faster at every batch; this one has linear_shrink and
    linear_expand."""

    def __init__(self, x, Wq, Ws, y, d_in=None, d_out=None):
        self.x, self.Wq, self.Ws, self.y = x, Wq, Ws, y
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_out = int(Wq.shape[0] if d_out is None else d_out)


class LinearI8IO:
    """One projection for linear_layer with an int8 base: x [rows, >= d_in]
    bf16, Wq int8 [d_out, >= d_in] (row stride a multiple of 16), Ws float32
    [d_out] (the scale of each output), y [rows, >= d_out] bf16 (written).
    Rows of x are quantised in the call."""

    def __init__(self, x, Wq, Ws, y, d_in=None, d_out=None):
        self.x, self.Wq, self.Ws, self.y = x, Wq, Ws, y
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_out = int(Wq.shape[0] if d_out is None else d_out)


class LinearQ4GIO:
    """One projection for linear_layer with a 4-bit base in groups of ``group``
    (32, 64 or 128) inputs: x [rows, >= d_in] bf16, Wq uint8 [d_out,
    >= d_in / 2] (packed as for LinearQ4IO, row stride a multiple of 16), Ws
    float32 [d_out, >= d_in / group], y [rows, >= d_out] bf16 (written).  Every
    projection of a call has the same group."""

    def __init__(self, x, Wq, Ws, y, group, d_in=None, d_out=None):
        self.x, self.Wq, self.Ws, self.y, self.group = x, Wq, Ws, y, int(group)
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_out = int(Wq.shape[0] if d_out is None else d_out)


def linear_q4g_workspace_bytes(num_rows: int, num_slots: int, max_rank: int, sum_d_in: int, n_modules: int) -> int:
    return int(lib().lora_linear_q4g_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n_modules))


class GatedIO:
    """The gate and up projections for gated_layer: x [rows, >= d_in], Wg and Wu
    [d_ff, >= d_in] (the base weights), h [rows, >= d_ff] (written), bf16."""

    def __init__(self, x, Wg, Wu, h, d_in=None, d_ff=None):
        self.x, self.Wg, self.Wu, self.h = x, Wg, Wu, h
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_ff = int(Wg.shape[0] if d_ff is None else d_ff)


class GatedQ4GIO:
    """The same with 4-bit base weights: Wgq, Wgs and Wuq, Wus as LinearQ4GIO's
    Wq, Ws."""

    def __init__(self, x, Wgq, Wgs, Wuq, Wus, h, group, d_in=None, d_ff=None):
        self.x, self.Wgq, self.Wgs, self.Wuq, self.Wus, self.h, self.group = x, Wgq, Wgs, Wuq, Wus, h, int(group)
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_ff = int(Wgq.shape[0] if d_ff is None else d_ff)


def gated_workspace_bytes(num_rows: int, num_slots: int, max_rank: int, d_in: int) -> int:
    return int(lib().lora_gated_workspace_bytes(num_rows, num_slots, max_rank, d_in))


def linear_i8_workspace_bytes(num_rows: int, num_slots: int, max_rank: int, sum_d_in: int, n_modules: int) -> int:
    return int(lib().lora_linear_i8_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n_modules))


def linear_workspace_bytes(num_rows: int, num_slots: int, max_rank: int, sum_d_in: int, n_modules: int) -> int:
    return int(lib().lora_linear_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n_modules))


_LIN_I8_PACK = struct.Struct("qqqqqqqii")
_LIN_Q4G_PACK = struct.Struct("qqqqqqqqiiii")
_GROUPED_PACK = struct.Struct("qqqqiiii")
assert _LIN_I8_PACK.size == ctypes.sizeof(_LinI8IO) and _GROUPED_PACK.size == ctypes.sizeof(_GroupedIO)


def _one_device(dev, tensors, what):
    """The call's device is the current one (its stream runs the kernels) and holds these tensors too."""
    import torch
    if dev != torch.cuda.current_device():
        raise ValueError(f"{what}: the tensors are on another device than the current one")
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"{what}: the tensors are on more than one device")


def _row_ids(row_adapter, num_rows):
    """The device of a call's row ids (int32, one per row)."""
    import torch
    if type(row_adapter) is not torch.Tensor or row_adapter.dtype is not torch.int32 or not row_adapter.is_cuda or \
            row_adapter.stride() != (1,):
        _need(row_adapter, torch.int32, "row_adapter", 1)
    if row_adapter.size(0) < num_rows:
        raise ValueError("row_adapter: fewer ids than num_rows")
    dev = row_adapter.get_device()
    if dev < 0:
        raise ValueError("row_adapter must be on the GPU")
    return dev


def _q4_weight(Wq, Ws, d_in, d_out, group, dev, name, fields):
    """(address, bytes per row, scales' address, scales per row) of a 4-bit weight."""
    import torch
    if group not in Q4_GROUPS:
        raise ValueError(f"{name}: group must be one of {Q4_GROUPS}")
    if d_in % group:
        raise ValueError(f"{name}: d_in must be a multiple of the group")
    wp, ldw = _rows(Wq, torch.uint8, d_out, d_in // 2, dev, name, fields[0])
    sp, lds = _rows(Ws, torch.float32, d_out, d_in // group, dev, name, fields[1])
    return wp, ldw, sp, lds


def _linear_q4g_array(ios, num_rows, row_adapter, rest):
    import torch
    bf16 = torch.bfloat16
    dev = _row_ids(row_adapter, num_rows)
    arr = (_LinQ4GIO * 7)()
    mask, group = 0, 0
    for i, name in enumerate(MODULES):
        io = ios.get(name)
        if io is None:
            continue
        if not isinstance(io, LinearQ4GIO):
            raise TypeError(_ONE_KIND)
        if group and io.group != group:
            raise ValueError("linear_layer: every projection has the same group")
        group = io.group
        xp, ldx = _rows(io.x, bf16, num_rows, io.d_in, dev, name, "x")
        yp, ldy = _rows(io.y, bf16, num_rows, io.d_out, dev, name, "y")
        weight = _q4_weight(io.Wq, io.Ws, io.d_in, io.d_out, group, dev, name, ("Wq", "Ws"))
        _LIN_Q4G_PACK.pack_into(arr, i * _LIN_Q4G_PACK.size, xp, ldx, *weight, yp, ldy, io.d_in, io.d_out, group, 0)
        mask |= 1 << i
    _one_device(dev, rest, "linear_layer")
    return arr, mask


def _linear_i8_array(ios, num_rows, row_adapter, rest):
    import torch
    bf16, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    if row_adapter.size(0) < num_rows:
        raise ValueError("row_adapter: fewer ids than num_rows")
    dev = row_adapter.get_device()
    if dev < 0:
        raise ValueError("row_adapter must be on the GPU")
    arr = (_LinI8IO * 7)()
    mask = 0
    for i, name in enumerate(MODULES):
        io = ios.get(name)
        if io is None:
            continue
        if not isinstance(io, LinearI8IO):
            raise TypeError(_ONE_KIND)
        Ws, d_out = io.Ws, io.d_out
        xp, ldx = _rows(io.x, bf16, num_rows, io.d_in, dev, name, "x")
        yp, ldy = _rows(io.y, bf16, num_rows, d_out, dev, name, "y")
        wp, ldw = _rows(io.Wq, i8, d_out, io.d_in, dev, name, "Wq")
        if Ws.dtype is not f32 or Ws.get_device() != dev or Ws.stride() != (1,):
            _need(Ws, f32, f"{name}.Ws", 1)
            _one_device(dev, (Ws,), name)
        if Ws.size(0) < d_out:
            raise ValueError(f"{name}.Ws: fewer scales than d_out")
        _LIN_I8_PACK.pack_into(arr, i * _LIN_I8_PACK.size, xp, ldx, wp, ldw, Ws.data_ptr(), yp, ldy, io.d_in, d_out)
        mask |= 1 << i
    _one_device(dev, rest, "linear_layer")
    return arr, mask


_LINEAR_KINDS = {LinearIO: (_LinIO, ""), LinearQ4IO: (_LinQ4IO, "_q4"), LinearI8IO: (_LinI8IO, "_i8"),
                 LinearQ4GIO: (_LinQ4GIO, "_q4g")}
_ONE_KIND = ("linear_layer: every projection LinearIO, or every projection LinearQ4IO, or every projection LinearI8IO, "
             "or every projection LinearQ4GIO")


def linear_layer(ios, num_rows, row_adapter, table, num_slots, seg, max_rank, ws, stream=None, module_mask=None,
                 _fn="lora_linear_layer"):
    """Base projection + delta of every projection in ``ios`` ({name:
    LinearIO}, or {name: LinearQ4IO} or {name: LinearQ4GIO} for 4-bit or
    {name: LinearI8IO} for int8 base weights); see lora_linear_layer,
    lora_linear_layer_q4, lora_linear_layer_q4g and lora_linear_layer_i8."""
    import torch
    if type(row_adapter) is not torch.Tensor or row_adapter.dtype is not torch.int32 or not row_adapter.is_cuda or \
            row_adapter.stride() != (1,):
        _need(row_adapter, torch.int32, "row_adapter", 1)
    # any object with its attributes is a bf16 projection, as for the other layer calls
    kind = next((k for k in (LinearQ4IO, LinearI8IO, LinearQ4GIO) if any(isinstance(io, k) for io in ios.values())), LinearIO)
    cstruct, suffix = _LINEAR_KINDS[kind]
    if kind is LinearI8IO or kind is LinearQ4GIO:
        _slot_table(table, num_slots, "table")
        array = _linear_i8_array if kind is LinearI8IO else _linear_q4g_array
        if kind is LinearQ4GIO and _fn != "lora_linear_layer":
            raise TypeError("linear_shrink, linear_expand: not for LinearQ4GIO")
        arr, mask = array(ios, num_rows, row_adapter, (table, ws, seg.perm))
        _fn += suffix
        _check(getattr(lib(), _fn)(arr, mask if module_mask is None else module_mask, num_rows, _ptr(row_adapter),
                                   _ptr(table), num_slots, seg.c(), max_rank, _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), _fn)
        return
    arr = (cstruct * 7)()
    mask = 0
    for i, name in enumerate(MODULES):
        io = ios.get(name)
        if io is None:
            continue
        if kind is not LinearIO and not isinstance(io, kind):
            raise TypeError(_ONE_KIND)
        for t, what in ((io.x, "x"), (io.y, "y")) + (((io.W, "W"),) if kind is LinearIO else ()):
            _need(t, torch.bfloat16, f"{name}.{what}", 2)
        if io.x.shape[0] < num_rows or io.y.shape[0] < num_rows:
            raise ValueError(f"{name}: fewer rows than num_rows")
        if kind is LinearQ4IO:
            _need(io.Wq, torch.uint8, f"{name}.Wq", 2)
            _need(io.Ws, torch.float32, f"{name}.Ws", 2)
            arr[i] = _LinQ4IO(io.x.data_ptr(), io.x.stride(0), io.Wq.data_ptr(), io.Wq.stride(0), io.Ws.data_ptr(),
                              io.Ws.stride(0), io.y.data_ptr(), io.y.stride(0), io.d_in, io.d_out)
        else:
            arr[i] = _LinIO(io.x.data_ptr(), io.x.stride(0), io.W.data_ptr(), io.W.stride(0), io.y.data_ptr(),
                            io.y.stride(0), io.d_in, io.d_out)
        mask |= 1 << i
    _fn += suffix
    _check(getattr(lib(), _fn)(arr, mask if module_mask is None else module_mask, num_rows, _ptr(row_adapter),
                               _ptr(table), num_slots, seg.c(), max_rank, _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)), _fn)


def linear_shrink(*args, **kw):
    """The shrink part of linear_layer (v per row and projection into ws)."""
    linear_layer(*args, _fn="lora_linear_shrink", **kw)


def linear_expand(*args, **kw):
    """The fused part of linear_layer (W.x + delta into y), after linear_shrink."""
    linear_layer(*args, _fn="lora_linear_expand", **kw)


def pack_table(A_ptrs, B_ptrs, ranks, scales, formats=None) -> np.ndarray:
    """Host bytes of a table of lora_adapter_entry_t; arrays of shape [num_slots, n_mod]
    (formats: FORMAT_BF16 where omitted)."""
    ranks = np.asarray(ranks)
    t = np.zeros(ranks.shape, TABLE_ENTRY_DTYPE)
    t["A"] = np.asarray(A_ptrs, np.uint64)
    t["B"] = np.asarray(B_ptrs, np.uint64)
    t["rank"] = ranks.astype(np.int32)
    t["scale"] = np.asarray(scales, np.float32)
    if formats is not None:
        t["format"] = np.asarray(formats, np.int32)
    return t


class GroupedIO:
    """One projection for grouped_layer: x [ceil(rows / rows_per_x), >= d_in]
    and y [rows, >= d_out], bf16; row b of the batch reads x row
    b // rows_per_x.  The weights come from the device table."""

    def __init__(self, x, y, d_in=None, d_out=None, rows_per_x: int = 1):
        self.x, self.y = x, y
        self.d_in = int(x.shape[1] if d_in is None else d_in)
        self.d_out = int(y.shape[1] if d_out is None else d_out)
        self.rows_per_x = int(rows_per_x)


def pack_weights(W_ptrs, ldw, Ws_ptrs=None) -> np.ndarray:
    """Host bytes of a table of lora_weight_entry_t; arrays of shape
    [num_slots, 7]: device addresses of the weights (0: none), elements per
    row, and for int8 weights the addresses of their output scales."""
    W = np.asarray(W_ptrs, np.uint64)
    t = np.zeros(W.shape, WEIGHT_ENTRY_DTYPE)
    t["W"] = W
    t["ldw"] = np.asarray(ldw, np.int64)
    if Ws_ptrs is not None:
        t["Ws"] = np.asarray(Ws_ptrs, np.uint64)
    return t


def grouped_workspace_bytes(num_rows: int, num_slots: int, sum_d_in: int, n_modules: int) -> int:
    return int(lib().lora_grouped_workspace_bytes(num_rows, num_slots, sum_d_in, n_modules))


def grouped_layer(ios, num_rows, weights, num_slots, seg, ws=None, stream=None, module_mask=None, int8=False):
    """Dense products grouped by slot of every projection in ``ios`` ({name:
    GroupedIO}): y[b] = W_a . x[b // rows_per_x] for the rows in a segment,
    W_a from the device table ``weights`` (pack_weights).  int8: the table's
    weights are int8 with output scales, rows of x are quantised in the call
    and ``ws`` is needed.  The tile follows num_rows over
    ``seg.max_segments`` (over num_slots where that is 0): state it when the
    batch uses few of the slots.  See lora_grouped_layer and
    lora_grouped_layer_i8."""
    import torch
    bf16 = torch.bfloat16
    arr = (_GroupedIO * 7)()
    mask = 0
    dev = weights.get_device()
    if dev < 0:
        raise ValueError("weights must be on the GPU")
    _slot_table(weights, num_slots, "weights")
    for i, name in enumerate(MODULES):
        io = ios.get(name)
        if io is None:
            continue
        fan = io.rows_per_x
        if fan < 1:
            raise ValueError(f"{name}: rows_per_x must be >= 1")
        xp, ldx = _rows(io.x, bf16, -(-num_rows // fan), io.d_in, dev, name, "x")
        yp, ldy = _rows(io.y, bf16, num_rows, io.d_out, dev, name, "y")
        _GROUPED_PACK.pack_into(arr, i * _GROUPED_PACK.size, xp, ldx, yp, ldy, io.d_in, io.d_out, fan, 0)
        mask |= 1 << i
    if module_mask is not None:
        mask = module_mask
    _one_device(dev, (seg.perm,) if ws is None else (seg.perm, ws), "grouped_layer")
    if int8:
        _check(lib().lora_grouped_layer_i8(arr, mask, num_rows, _ptr(weights), num_slots, seg.c(), _ptr(ws),
                                           0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
               "lora_grouped_layer_i8")
    else:
        _check(lib().lora_grouped_layer(arr, mask, num_rows, _ptr(weights), num_slots, seg.c(), _stream(stream)),
               "lora_grouped_layer")


def _activation(name) -> int:
    try:
        return ACTIVATIONS.index(name)
    except ValueError:
        raise ValueError(f"activation must be one of {ACTIVATIONS}") from None


def gated_layer(io, num_rows, row_adapter, table, num_slots, seg, max_rank, ws, stream=None, activation="silu"):
    """The gated half of a feed-forward block: h = act(gate) * up, both
    projections with the rows' adapters (table columns "gate" and "up").  ``io``:
    GatedIO, or GatedQ4GIO for 4-bit base weights; ``activation``: one of
    ACTIVATIONS; ``ws``: gated_workspace_bytes.  See lora_gated_layer and
    lora_gated_layer_q4g."""
    import torch
    bf16 = torch.bfloat16
    act = _activation(activation)
    dev = _row_ids(row_adapter, num_rows)
    _slot_table(table, num_slots, "table")
    xp, ldx = _rows(io.x, bf16, num_rows, io.d_in, dev, "gated_layer", "x")
    hp, ldh = _rows(io.h, bf16, num_rows, io.d_ff, dev, "gated_layer", "h")
    if isinstance(io, GatedQ4GIO):
        gate = _q4_weight(io.Wgq, io.Wgs, io.d_in, io.d_ff, io.group, dev, "gated_layer", ("Wgq", "Wgs"))
        up = _q4_weight(io.Wuq, io.Wus, io.d_in, io.d_ff, io.group, dev, "gated_layer", ("Wuq", "Wus"))
        arg, fn = _GatedQ4GIO(xp, ldx, *gate, *up, hp, ldh, io.d_in, io.d_ff, io.group, 0), "lora_gated_layer_q4g"
    else:
        gate = _rows(io.Wg, bf16, io.d_ff, io.d_in, dev, "gated_layer", "Wg")
        up = _rows(io.Wu, bf16, io.d_ff, io.d_in, dev, "gated_layer", "Wu")
        arg, fn = _GatedIO(xp, ldx, *gate, *up, hp, ldh, io.d_in, io.d_ff), "lora_gated_layer"
    _one_device(dev, (table, ws, seg.perm), "gated_layer")
    _check(getattr(lib(), fn)(arg, act, num_rows, _ptr(row_adapter), _ptr(table), num_slots, seg.c(), max_rank, _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), fn)


def pack_weights_q4g(W_ptrs, ldw, Ws_ptrs, lds) -> np.ndarray:
    """Host bytes of a table of lora_weight_q4g_entry_t; arrays of shape
    [num_slots, 7]: device addresses of the packed weights (0: none), bytes per
    row, addresses of their group scales, floats per row of those."""
    W = np.asarray(W_ptrs, np.uint64)
    t = np.zeros(W.shape, WEIGHT_Q4G_ENTRY_DTYPE)
    t["W"] = W
    t["ldw"] = np.asarray(ldw, np.int64)
    t["Ws"] = np.asarray(Ws_ptrs, np.uint64)
    t["lds"] = np.asarray(lds, np.int64)
    return t


_GATE = MODULES.index("gate")


def _grouped_array(ios, num_rows, weights, num_slots, seg, what):
    import torch
    bf16 = torch.bfloat16
    arr = (_GroupedIO * 7)()
    mask = 0
    dev = weights.get_device()
    if dev < 0:
        raise ValueError("weights must be on the GPU")
    _slot_table(weights, num_slots, "weights")
    for i, name in enumerate(MODULES):
        io = ios.get(name)
        if io is None:
            continue
        fan = io.rows_per_x
        if fan < 1:
            raise ValueError(f"{name}: rows_per_x must be >= 1")
        xp, ldx = _rows(io.x, bf16, -(-num_rows // fan), io.d_in, dev, name, "x")
        yp, ldy = _rows(io.y, bf16, num_rows, io.d_out, dev, name, "y")
        _GROUPED_PACK.pack_into(arr, i * _GROUPED_PACK.size, xp, ldx, yp, ldy, io.d_in, io.d_out, fan, 0)
        mask |= 1 << i
    if seg.perm.size(0) < num_rows:  # the kernels read the segments beside their number: as many as the rows could have
        raise ValueError("Segments buffers too small for this batch")
    _one_device(dev, (seg.perm,), what)
    return arr, mask


def grouped_layer_q4g(ios, num_rows, weights, num_slots, seg, group, stream=None, module_mask=None):
    """grouped_layer with 4-bit weights and a scale per group of ``group`` (32, 64
    or 128) inputs from the device table ``weights`` (pack_weights_q4g); see
    lora_grouped_layer_q4g."""
    arr, mask = _grouped_array(ios, num_rows, weights, num_slots, seg, "grouped_layer_q4g")
    _check(lib().lora_grouped_layer_q4g(arr, mask if module_mask is None else module_mask, num_rows, _ptr(weights), num_slots,
                                        group, seg.c(), _stream(stream)), "lora_grouped_layer_q4g")


def grouped_gated_layer(io, num_rows, weights, num_slots, seg, stream=None, activation="silu"):
    """The gated half of a feed-forward block with a whole gate and up weight per
    slot: io.y[b] = act(Wg_a . x) * (Wu_a . x), x = io.x[b // rows_per_x], for the
    rows in a segment.  ``io``: GroupedIO whose y is h; ``weights``: the device
    table (pack_weights), columns "gate" and "up".  State ``seg.max_segments`` as
    for grouped_layer.  See lora_grouped_gated_layer."""
    act = _activation(activation)
    arr, _ = _grouped_array({"gate": io}, num_rows, weights, num_slots, seg, "grouped_gated_layer")
    _check(lib().lora_grouped_gated_layer(arr[_GATE], act, num_rows, _ptr(weights), num_slots, seg.c(), _stream(stream)),
           "lora_grouped_gated_layer")


def grouped_gated_layer_q4g(io, num_rows, weights, num_slots, seg, group, stream=None, activation="silu"):
    """grouped_gated_layer with 4-bit weights (pack_weights_q4g); see
    lora_grouped_gated_layer_q4g."""
    act = _activation(activation)
    arr, _ = _grouped_array({"gate": io}, num_rows, weights, num_slots, seg, "grouped_gated_layer_q4g")
    _check(lib().lora_grouped_gated_layer_q4g(arr[_GATE], act, num_rows, _ptr(weights), num_slots, group, seg.c(), _stream(stream)),
           "lora_grouped_gated_layer_q4g")


def build_segments(row_adapter, num_slots: int, seg: Segments, ws, stream=None):
    """Group rows by adapter slot (stable); see lora_build_segments."""
    import torch
    if type(row_adapter) is not torch.Tensor or row_adapter.dtype is not torch.int32 or not row_adapter.is_cuda or \
            row_adapter.stride() != (1,):
        _need(row_adapter, torch.int32, "row_adapter", 1)
    n = row_adapter.size(0)
    if n > seg.num_rows:
        raise ValueError("Segments buffers too small for this batch")
    _check(lib().lora_build_segments(_ptr(row_adapter), n, num_slots, seg.c(), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream)), "lora_build_segments")


def shrink(x, table, num_slots: int, n_mod: int, module: int, seg: Segments, max_rank: int, v, ws, stream=None):
    """v[b, :rank] = A . x[b] for rows in a segment; see lora_shrink."""
    import torch
    _need(x, torch.bfloat16, "x", 2)
    _need(v, torch.float32, "v", 2)
    _check(lib().lora_shrink(_ptr(x), x.stride(0), x.shape[0], x.shape[1], _ptr(table), num_slots, n_mod, module,
                             seg.c(), max_rank, _ptr(v), v.stride(0), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(stream)), "lora_shrink")


def expand(v, table, num_slots: int, n_mod: int, module: int, seg: Segments, max_rank: int, y, ws, stream=None):
    """y[b] = bf16(y[b] + scale * B . v[b]) for rows in a segment; see lora_expand."""
    import torch
    _need(v, torch.float32, "v", 2)
    _need(y, torch.bfloat16, "y", 2)
    _check(lib().lora_expand(_ptr(v), v.stride(0), y.shape[0], y.shape[1], _ptr(table), num_slots, n_mod, module,
                             seg.c(), max_rank, _ptr(y), y.stride(0), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(stream)), "lora_expand")


def _ios(ios, num_rows):
    import torch
    arr = (_IO * 7)()
    mask = 0
    for i, name in enumerate(MODULES):
        io = ios.get(name) if isinstance(ios, dict) else (ios[i] if i < len(ios) else None)
        if io is None:
            continue
        _need(io.x, torch.bfloat16, f"{name}.x", 2)
        _need(io.y, torch.bfloat16, f"{name}.y", 2)
        if io.x.shape[0] < num_rows or io.y.shape[0] < num_rows:
            raise ValueError(f"{name}: fewer rows than num_rows")
        arr[i] = _IO(io.x.data_ptr(), io.x.stride(0), io.y.data_ptr(), io.y.stride(0), io.d_in, io.d_out)
        mask |= 1 << i
    return arr, mask


MASK_INT8_ITEMS = 1 << 16  # LORA_MASK_INT8_ITEMS


def module_mask(ios, int8_items: bool = False) -> int:
    """The module_mask of the projections in ``ios`` ({name: io}); with
    int8_items, LORA_MASK_INT8_ITEMS too (the table's entries are int8: the
    shrink's items are sized for one-byte factors)."""
    mask = 0
    for i, name in enumerate(MODULES):
        if name in ios:
            mask |= 1 << i
    return mask | (MASK_INT8_ITEMS if int8_items else 0)


def _layer(fn, what, ios, num_rows, table, num_slots, seg, max_rank, ws, stream, module_mask):
    arr, mask = _ios(ios, num_rows)
    if module_mask is None:
        module_mask = mask
    _check(fn(arr, module_mask, num_rows, _ptr(table), num_slots, seg.c(), max_rank, _ptr(ws),
              ws.numel() * ws.element_size(), _stream(stream)), what)


def apply_layer(ios, num_rows, table, num_slots, seg, max_rank, ws, stream=None, module_mask=None):
    """Delta of every projection given in ``ios`` ({name: ModuleIO}); see lora_apply_layer."""
    _layer(lib().lora_apply_layer, "lora_apply_layer", ios, num_rows, table, num_slots, seg, max_rank, ws, stream,
           module_mask)


def decode_layer(ios, num_rows, row_adapter, table, num_slots, seg, max_rank, ws, stream=None, module_mask=None):
    """Segments and the layer delta of a decode batch (one launch for a batch
    of distinct adapters); see lora_decode_layer."""
    import torch
    _need(row_adapter, torch.int32, "row_adapter", 1)
    if row_adapter.shape[0] < num_rows:
        raise ValueError("row_adapter: fewer ids than num_rows")
    arr, mask = _ios(ios, num_rows)
    if module_mask is None:
        module_mask = mask
    _check(lib().lora_decode_layer(arr, module_mask, num_rows, _ptr(row_adapter), _ptr(table), num_slots, seg.c(),
                                   max_rank, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "lora_decode_layer")


def decode_layer_launches(ios, num_rows, num_slots, seg, max_rank, module_mask=None) -> int:
    """Kernel launches lora_decode_layer makes for these arguments (1 or 3; 0 if it would reject them)."""
    arr, mask = _ios(ios, num_rows)
    return int(lib().lora_decode_layer_launches(arr, mask if module_mask is None else module_mask, num_rows,
                                                num_slots, seg.c(), max_rank))


def apply_layer_noalloc(ios, num_rows, table, num_slots, seg, max_rank, stream=None, module_mask=None):
    """apply_layer with the library's static device scratch instead of a
    workspace (allocates nothing); see lora_apply_layer_noalloc."""
    arr, mask = _ios(ios, num_rows)
    if module_mask is None:
        module_mask = mask
    _check(lib().lora_apply_layer_noalloc(arr, module_mask, num_rows, _ptr(table), num_slots, seg.c(), max_rank,
                                          _stream(stream)), "lora_apply_layer_noalloc")


def layer_shrink(ios, num_rows, table, num_slots, seg, max_rank, ws, stream=None, module_mask=None):
    _layer(lib().lora_layer_shrink, "lora_layer_shrink", ios, num_rows, table, num_slots, seg, max_rank, ws, stream,
           module_mask)


def layer_expand(ios, num_rows, table, num_slots, seg, max_rank, ws, stream=None, module_mask=None):
    _layer(lib().lora_layer_expand, "lora_layer_expand", ios, num_rows, table, num_slots, seg, max_rank, ws, stream,
           module_mask)


def apply_layer_stacked(ios, num_rows, row_adapters, table, num_slots, seg, max_rank, ws, stream=None,
                        module_mask=None, pass_max_rank=None):
    """Several adapters per row (``row_adapters``: device int32 [num_rows, depth],
    -1 pads; ``pass_max_rank``: optional largest rank of each column); see
    lora_apply_layer_stacked."""
    import torch
    _need(row_adapters, torch.int32, "row_adapters", 2)
    if row_adapters.shape[0] < num_rows or not row_adapters.is_contiguous():
        raise ValueError("row_adapters: a contiguous [num_rows, depth] tensor")
    depth = row_adapters.shape[1]
    pr = None
    if pass_max_rank is not None:
        pr = np.ascontiguousarray(pass_max_rank, dtype=np.int32)
        if pr.shape != (depth,):
            raise ValueError("pass_max_rank: one rank per column")
    arr, mask = _ios(ios, num_rows)
    if module_mask is None:
        module_mask = mask
    _check(lib().lora_apply_layer_stacked(arr, module_mask, num_rows, _ptr(row_adapters), depth,
                                          None if pr is None else pr.ctypes.data_as(ctypes.c_void_p),
                                          _ptr(table), num_slots, seg.c(), max_rank, _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)),
           "lora_apply_layer_stacked")


def form_batch(adapters, max_batch: int, max_distinct: int, min_batch: int = 0, reserved_tail: int = 0,
               waited_ms=None, max_wait_ms: float = 0.0) -> np.ndarray:
    """lora_form_batch on host arrays: queue positions of the chosen requests,
    in batch order.  ``adapters``: int32 adapter slot per waiting request,
    oldest first (negative = base only); ``waited_ms``: optional float ages."""
    a = np.ascontiguousarray(adapters, dtype=np.int32)
    w = None if waited_ms is None else np.ascontiguousarray(waited_ms, dtype=np.float32)
    if w is not None and w.shape != a.shape:
        raise LoraError("form_batch: waited_ms must match adapters")
    out = np.empty(max(1, min(int(max_batch), a.size)), np.int32)
    count = ctypes.c_int32(0)
    code = host_lib().lora_form_batch(a.ctypes.data_as(ctypes.c_void_p), a.size,
                                 None if w is None else w.ctypes.data_as(ctypes.c_void_p), float(max_wait_ms),
                                 int(max_batch), int(max_distinct), int(min_batch), int(reserved_tail),
                                 out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(count))
    _check(code, "form_batch")
    return out[:count.value].copy()
