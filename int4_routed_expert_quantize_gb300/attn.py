"""Binding of the paged-cache attention in libcoli_moe.so (include/coli_attn.h).

    eng = attn.PagedAttention(n_q=48, n_kv=8, head_dim=128, page=64, max_tokens=512, max_seqs=64)
    cache = eng.bind_cache(k_cache, v_cache)           # [pages, n_kv, page, head_dim], any strides
    batch = attn.Batch(q_start, kv_len, table, n_tokens=T, max_q=1)
    q = eng.append(cache, batch, k, v, q)              # rotate, store, return the rotated queries
    o = eng.window(cache, batch, q, window=4096, sinks=4)
    o = eng.prefix(cache, batch, prefix_table, prefix_len, q)

Argument marshalling only (the three calls' in _attn_py, csrc/attn_py.cpp); every step runs in the library's CUDA
kernels.
"""
import ctypes
import math
import sys

import torch

from . import coli

_i, _f, _vp, _i64, _d = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64, ctypes.c_double

DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class AttnConfig(ctypes.Structure):
    _fields_ = [("n_q", _i), ("n_kv", _i), ("head_dim", _i), ("page", _i), ("dtype", _i),
                ("max_tokens", _i), ("max_seqs", _i), ("rot_dim", _i), ("rot_interleaved", _i),
                ("rope_base", _d), ("inv_freq", ctypes.POINTER(_d))]


class AttnCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("n_pages", _i64), ("k_page_stride", _i64), ("k_head_stride", _i64),
                ("k_slot_stride", _i64), ("v_page_stride", _i64), ("v_head_stride", _i64),
                ("v_slot_stride", _i64)]


class AttnBatch(ctypes.Structure):
    _fields_ = [("q_start", _vp), ("kv_len", _vp), ("table", _vp), ("table_stride", _i64), ("n_seqs", _i),
                ("max_pages", _i), ("n_tokens", _i), ("max_q", _i)]


class BatchArgs(ctypes.Structure):  # csrc/attn_py.cpp
    _anonymous_ = ("batch",)
    _fields_ = [("batch", AttnBatch), ("device", _i)]


class Engine(ctypes.Structure):  # csrc/attn_py.cpp
    _fields_ = [("handle", _vp), ("n_q", _i), ("n_kv", _i), ("head_dim", _i), ("dtype", _i), ("device", _i),
                ("scale", _f)]


_lib = _calls = None


def lib():
    global _lib, _calls
    L = coli.lib()
    if _lib is not L:
        L.coli_attn_create.argtypes = [ctypes.POINTER(AttnConfig), ctypes.POINTER(_vp)]
        L.coli_attn_destroy.argtypes = [_vp]
        L.coli_attn_destroy.restype = None
        L.coli_attn_cache_bind.argtypes = [_vp, ctypes.POINTER(AttnCache), ctypes.POINTER(_vp)]
        L.coli_attn_cache_release.argtypes = [_vp]
        L.coli_attn_cache_release.restype = None
        L.coli_attn_append.argtypes = [_vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp]
        L.coli_attn_window.argtypes = [_vp, _vp, _vp, _vp, _i64, _i, _i, _f, _vp, _i64, _vp, _vp]
        L.coli_attn_prefix.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _vp, _i64, _f, _vp, _i64, _vp, _vp]
        L.coli_attn_status.argtypes = [_vp, _vp]
        L.coli_attn_launches.argtypes = [_vp, _i, _i]
        from . import _attn_py
        _lib, _calls = L, _attn_py
    return L


def _int32(t, dims, what):
    if t.dtype is not torch.int32 or t.dim() != dims or (t.numel() and t.stride(-1) != 1) or not t.is_cuda:
        raise ValueError(f"{what}: a {dims}-dimensional int32 tensor on the device, rows contiguous")
    return t


def _row_stride(table):
    """elements between the rows of a page table; 0: an expanded row, which all sequences share"""
    rows, width = table.shape
    if rows < 2:  # one row has no stride of its own
        return width
    if 0 < table.stride(0) < width:
        raise ValueError("table: rows that overlap")
    return table.stride(0)


class Batch:
    """The ragged batch of a call: sequence b has the query tokens q_start[b] .. q_start[b+1]-1, the last
    of its kv_len[b] cached tokens, whose pages are table[b] (rows may be slices of wider ones, or one row
    expanded).  The three int32 tensors stay the caller's (they may be updated in place between calls and are
    read on the device); n_tokens is the number of query tokens, max_q at least the new tokens of any sequence."""

    def __init__(self, q_start, kv_len, table, n_tokens, max_q):
        _int32(q_start, 1, "q_start"), _int32(kv_len, 1, "kv_len"), _int32(table, 2, "table")
        n = kv_len.shape[0]
        if q_start.shape[0] != n + 1 or table.shape[0] != n:
            raise ValueError("q_start has one entry more than kv_len, table one row for each sequence")
        self.q_start, self.kv_len, self.table = q_start, kv_len, table
        self.n_tokens, self.max_q, self.n_seqs = int(n_tokens), int(max_q), n
        if not q_start.device == kv_len.device == table.device:
            raise ValueError("q_start, kv_len and table are on one device")
        self.c = BatchArgs(AttnBatch(q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), _row_stride(table), n,
                                     table.shape[1], self.n_tokens, self.max_q), table.device.index)
        self.ref = ctypes.addressof(self.c)


class KvCache:
    """A cache bound to an engine (coli_attn_cache_bind); keeps the two tensors alive."""

    def __init__(self, engine, k, v):
        dims = (engine.n_kv, engine.page, engine.head_dim)
        for t in (k, v):
            if t.dim() != 4 or tuple(t.shape[1:]) != dims or t.dtype is not engine.dtype or not t.is_cuda or \
                    t.device.index != engine.device:
                raise ValueError(f"the cache is [pages, {dims[0]}, {dims[1]}, {dims[2]}] of {engine.dtype} on the "
                                 "engine's device")
            if t.stride(3) != 1:
                raise ValueError("a head's values are contiguous")
        if k.shape[0] != v.shape[0]:
            raise ValueError("K and V have the same number of pages")
        self.k, self.v = k, v

        def strides(t):  # a dimension of one has no stride of its own
            return [t.stride(i) if t.shape[i] > 1 else max(t.stride(i), engine.head_dim) // 8 * 8 for i in range(3)]

        c = AttnCache(k.data_ptr(), v.data_ptr(), k.shape[0], *strides(k), *strides(v))
        h = _vp()
        coli._check(lib().coli_attn_cache_bind(engine.h, ctypes.byref(c), ctypes.byref(h)), "coli_attn_cache_bind")
        self.h = h
        self.ref = h.value

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            lib().coli_attn_cache_release(self.h)
            self.h, self.ref = _vp(), 0

    def __del__(self):
        if sys.is_finalizing():  # the process is exiting: no native calls during teardown
            return
        try:
            self.close()
        except Exception:
            pass


def _handle(stream):
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _done(out, given, stream, what):
    """a call's output, or the error that its status stands for; a new output made on another stream than the
    current one is kept from reuse there until the current one is done with it"""
    if out.__class__ is int:
        raise coli.ColiError(out, what)
    if given is None and out is not None and stream is not None:
        out.record_stream(torch.cuda.current_stream(out.device))
    return out


class PagedAttention:
    """Shapes, rotation and workspace of the attention over a paged cache on the current device.
    rot_dim None rotates the whole head, 0 none of it; inv_freq (rot_dim/2 radians per position) takes
    the place of rope_base.  A call's `stream` (a torch stream or a handle; the current one by default) has to have
    waited for what writes its tensors; a new output is that stream's memory, for others to read once they have
    waited for it."""

    def __init__(self, n_q, n_kv, head_dim, page, max_tokens, max_seqs, dtype=torch.bfloat16, rot_dim=None,
                 interleaved=False, rope_base=10000.0, inv_freq=None):
        if dtype not in DTYPES:
            raise ValueError(f"{dtype}: the attention kernels take bfloat16 or float16")
        rot = head_dim if rot_dim is None else rot_dim
        freq = None
        if inv_freq is not None:
            freq = (_d * len(inv_freq))(*[float(x) for x in inv_freq])
            if len(inv_freq) != rot // 2:
                raise ValueError(f"inv_freq has rot_dim/2 = {rot // 2} entries")
        cfg = AttnConfig(n_q, n_kv, head_dim, page, DTYPES[dtype], max_tokens, max_seqs, rot, int(interleaved),
                         rope_base, freq)
        h = _vp()
        coli._check(lib().coli_attn_create(ctypes.byref(cfg), ctypes.byref(h)), "coli_attn_create")
        self.h = h
        self.n_q, self.n_kv, self.head_dim, self.page, self.dtype = n_q, n_kv, head_dim, page, dtype
        self.max_tokens, self.max_seqs, self.rot_dim = max_tokens, max_seqs, rot
        self.scale = 1.0 / math.sqrt(head_dim)
        self.device = torch.cuda.current_device()
        self.c = Engine(h, n_q, n_kv, head_dim, DTYPES[dtype], self.device, self.scale)
        self.ref = ctypes.addressof(self.c)

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            lib().coli_attn_destroy(self.h)
            self.h = self.c.handle = _vp()

    __del__ = KvCache.__del__

    def bind_cache(self, k_cache, v_cache):
        return KvCache(self, k_cache, v_cache)

    def append(self, cache, batch, k, v, q=None, q_out=None, pos_base=None, stream=None):
        """Stores the batch's new keys (rotated) and values in the cache; rotates q into q_out (new by
        default, q itself for in place) and returns it.  k, v [n_tokens, n_kv, head_dim] and q [n_tokens, n_q,
        head_dim] may be slices of a wider row.  pos_base: int32 [1] on the device, added to the positions
        for the rotation (the length of a shared prefix).  coli_attn_append"""
        out = _calls.append(self.ref, cache.ref, batch.ref, k, v, q, q_out, pos_base,
                            stream if stream is None else _handle(stream))
        return out if stream is None and out.__class__ is not int else _done(out, q_out, stream, "coli_attn_append")

    def window(self, cache, batch, q, window=-1, sinks=0, scale=None, out=None, lse=None, stream=None):
        """Causal attention over the last `window` keys (all with -1) and the first `sinks` ones ->
        [n_tokens, n_q, head_dim]; lse: float32 [n_tokens, n_q] to fill, or None.  coli_attn_window"""
        o = _calls.window(self.ref, cache.ref, batch.ref, q, window, sinks, scale, out, lse,
                          stream if stream is None else _handle(stream))
        return o if stream is None and o.__class__ is not int else _done(o, out, stream, "coli_attn_window")

    def prefix(self, cache, batch, prefix_table, prefix_len, q, scale=None, out=None, lse=None, stream=None):
        """Attention of a batch behind a shared prefix: prefix_len (int32 [1] on the device) tokens in the
        pages prefix_table (int32 [pages]), then each sequence's own cache.  coli_attn_prefix"""
        o = _calls.prefix(self.ref, cache.ref, batch.ref, prefix_table, prefix_len, q, scale, out, lse,
                          stream if stream is None else _handle(stream))
        return o if stream is None and o.__class__ is not int else _done(o, out, stream, "coli_attn_prefix")

    def status(self, stream=None):
        """device status of earlier calls (coli_attn_status); 0 when all went well"""
        return int(lib().coli_attn_status(self.h, coli._stream(stream)))

    def launches(self, op, n_seqs):
        """kernels one call launches at most, with n_seqs sequences; op "append", "window" or "prefix" (coli_attn_launches)"""
        n = int(lib().coli_attn_launches(self.h, ("append", "window", "prefix").index(op), n_seqs))
        if n < 0:
            raise coli.ColiError(n, "coli_attn_launches")
        return n
