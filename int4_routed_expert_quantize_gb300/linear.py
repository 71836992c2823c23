"""Binding of the 4-bit products for few tokens in libcoli_moe.so (include/coli_linear.h).

    packed, scales = linear.quantize(w, group=128)            # w [rows, cols] on the device -> 4-bit codes, bfloat16 scales
    proj = linear.Int4Linear(packed, scales, max_tokens=16)   # the library's own copy; the tensors may go
    y = proj.forward(x)                                       # [tokens, cols] -> [tokens, rows]

Argument marshalling only (the call's in _attn_py, csrc/attn_py.cpp); every step runs in the library's CUDA kernels.
"""
import ctypes

import torch

from . import attn, coli

_i, _vp, _i64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_int64

DTYPES = attn.DTYPES


class LinearConfig(ctypes.Structure):
    _fields_ = [("rows", _i), ("cols", _i), ("group", _i), ("dtype", _i), ("max_tokens", _i)]


class Weights(ctypes.Structure):  # csrc/attn_py.cpp
    _fields_ = [("handle", _vp), ("rows", _i), ("cols", _i), ("dtype", _i), ("device", _i)]


_lib = None


def lib():
    global _lib
    L = attn.lib()
    if _lib is not L:
        L.coli_linear_create.argtypes = [ctypes.POINTER(LinearConfig), ctypes.POINTER(_vp)]
        L.coli_linear_destroy.argtypes = [_vp]
        L.coli_linear_destroy.restype = None
        L.coli_linear_load.argtypes = [_vp, _vp, _vp, _vp]
        L.coli_linear_forward.argtypes = [_vp, _vp, _i64, _i, _vp, _i64, _vp]
        L.coli_linear_status.argtypes = [_vp, _vp]
        L.coli_linear_quantize.argtypes = [_vp, _i64, _i, _i, _i, _vp, _vp, _vp]
        _lib = L
    return L


def quantize(w, group=128, dtype=torch.bfloat16, stream=None):
    """w float32 [rows, cols] on the current device -> codes uint8 [rows, cols/2], scales of dtype [rows, cols/group], in memory
    of `stream` (the current one by default), for others to read once they have waited for it.  coli_linear_quantize"""
    if w.dtype is not torch.float32 or w.dim() != 2 or not w.is_contiguous() or not w.is_cuda or \
            w.device.index != torch.cuda.current_device():
        raise ValueError("w: contiguous float32 [rows, cols] on the current device")
    if dtype not in DTYPES:
        raise ValueError(f"{dtype}: scales are bfloat16 or float16")
    if group not in (32, 64, 128) or w.shape[1] % group or w.shape[1] == 0:
        raise ValueError("groups of 32, 64 or 128 columns divide the columns")
    rows, cols = w.shape
    if stream is not None and not isinstance(stream, torch.cuda.Stream):  # a handle; 0 and 1 are the default stream's
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) > 1 else torch.cuda.default_stream()
    with torch.cuda.stream(stream):  # None: nothing changes
        packed = torch.empty((rows, cols // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((rows, cols // group), dtype=dtype, device=w.device)
    coli._check(lib().coli_linear_quantize(w.data_ptr(), rows, cols, group, DTYPES[dtype], packed.data_ptr(), scales.data_ptr(),
                                           coli._stream(stream)), "coli_linear_quantize")
    if stream is not None:  # kept from reuse there until the current stream is done with them
        packed.record_stream(torch.cuda.current_stream()), scales.record_stream(torch.cuda.current_stream())
    return packed, scales


class Int4Linear:
    """Weights of y = W x on the current device: packed uint8 [rows, cols/2] (two's-complement nibbles, the even column low) and scales
    bfloat16 or float16 [rows, cols/group], which is the type of x and y.  Both are copied into the library's layout; `stream` (the
    current one by default) has to have waited for what writes them."""

    def __init__(self, packed, scales, max_tokens, stream=None):
        if scales.dtype not in DTYPES:
            raise ValueError(f"{scales.dtype}: scales are bfloat16 or float16")
        device = torch.cuda.current_device()
        for t, kind, what in ((packed, torch.uint8, "packed"), (scales, scales.dtype, "scales")):
            if t.dim() != 2 or t.dtype is not kind or not t.is_contiguous() or not t.is_cuda or t.device.index != device:
                raise ValueError(f"{what}: a contiguous 2-dimensional {kind} tensor on the current device")
        rows, cols = packed.shape[0], 2 * packed.shape[1]
        if scales.shape[0] != rows or scales.shape[1] < 1 or cols % scales.shape[1]:
            raise ValueError("scales: one for each row and group of columns")
        self.rows, self.cols, self.group, self.dtype = rows, cols, cols // scales.shape[1], scales.dtype
        self.max_tokens, self.device = max_tokens, device
        cfg = LinearConfig(rows, cols, self.group, DTYPES[self.dtype], max_tokens)
        h = _vp()
        coli._check(lib().coli_linear_create(ctypes.byref(cfg), ctypes.byref(h)), "coli_linear_create")
        self.h = h
        coli._check(lib().coli_linear_load(h, packed.data_ptr(), scales.data_ptr(), coli._stream(stream)), "coli_linear_load")
        self.c = Weights(h, rows, cols, DTYPES[self.dtype], device)
        self.ref = ctypes.addressof(self.c)

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            lib().coli_linear_destroy(self.h)
            self.h = _vp()
            if hasattr(self, "c"):
                self.c.handle = _vp()

    __del__ = attn.KvCache.__del__

    def forward(self, x, out=None, stream=None):
        """x [tokens, cols] (rows may be slices of wider ones) -> out [tokens, rows], new by default.  coli_linear_forward"""
        y = attn._calls.linear(self.ref, x, out, stream if stream is None else attn._handle(stream))
        return y if stream is None and y.__class__ is not int else attn._done(y, out, stream, "coli_linear_forward")

    def status(self, stream=None):
        """device status of earlier calls (coli_linear_status); 0 when all went well"""
        return int(lib().coli_linear_status(self.h, coli._stream(stream)))
