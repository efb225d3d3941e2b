"""MI355X (gfx950) multi-buffer all-reduce core: Python binding of libarcore.

A thin ctypes layer over the C-ABI in ``include/ar.h``.  Every function has
the C name and only marshals arguments: torch tensors become device
pointers and element counts, torch streams become ``hipStream_t`` handles.
All arithmetic runs in the HIP kernels of ``libarcore.so``; there is no
fallback of any kind.  If the library is missing, every call raises.

``prepare(func, *args, **kwargs)`` runs a device call's checks and
marshalling once and returns a handle that makes the same C-ABI call each
time it is called: for loops that pass the same buffers on every step.

bf16 buffers may be passed as ``torch.bfloat16`` or ``torch.int16`` /
``torch.uint16`` tensors (only the 16-bit patterns matter); payload words as
``torch.int64`` / ``torch.uint64`` tensors; error records as a 2-element
64-bit tensor.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Sequence

__all__ = [
    "ARError", "Prepared", "prepare", "lib", "lib_path", "ar_status_str", "ar_version", "ar_reduce_oneshot",
    "ar_reduce_2stage", "ar_reduce_2stage_static", "ar_pack_fused", "ar_unpack_fused", "ar_rd_schedule",
    "ar_reduce_ubatch", "ar_err_init", "rd_mailbox_words",
    "AR_OK", "AR_ERR_INVALID", "AR_ERR_ALIGN", "AR_ERR_ALIAS", "AR_ERR_UNSUPPORTED",
    "AR_ERR_HIP", "AR_ERR_SIZE", "AR_STATIC_SCRATCH_ELEMS", "AR_MAX_RANKS", "AR_VARIANT_ONESHOT", "AR_VARIANT_2STAGE", "AR_UBATCH_BOUNDED",
    "AR_RD_STAGED", "AR_RD_FP32_CARRY", "ar_set_launch_shape", "ar_get_launch_shape",
    "AR_KERNEL_ONESHOT", "AR_KERNEL_2STAGE", "AR_KERNEL_UBATCH", "AR_KERNEL_RS", "AR_KERNEL_AG",
    "AR_KERNEL_PACK", "AR_KERNEL_UNPACK", "AR_KERNEL_RD", "AR_KERNEL_RDSTEP", "AR_KERNEL_UNPACK_WAIT",
    "AR_KERNEL_UBATCH_FLAGS", "ar_unpack_fused_wait", "ar_reduce_ubatch_flags", "ubatch_chunk_count",
    "AR_KERNEL_QUANT_FP8", "AR_KERNEL_REDUCE_FP8", "AR_KERNEL_REDUCE_FP8_ALL", "ar_quantize_fp8", "ar_reduce_fp8", "fp8_scale_count",
    "AR_KERNEL_ONESHOT_SMALL", "AR_KERNEL_2STAGE_SMALL", "AR_KERNEL_RD_SMALL", "AR_KERNEL_RDSTEP_SMALL",
    "AR_KERNEL_PACK_SMALL", "AR_KERNEL_UNPACK_SMALL", "AR_KERNEL_UBATCH_BOUNDED",
    "AR_KERNEL_2STAGE_INPLACE_SMALL",
    "AR_SMALL_ELEMS",
    "FP8_BLOCK",
    "ar_reduce_norm", "ar_norm_bwd", "ar_quantize_block", "ar_gemm_fp8", "norm_bwd_workspace", "gemm_fp8_workspace",
    "fp8_codes_empty", "fp8_scales_empty",
    "AR_BLOCK", "AR_SCALE_F32", "AR_SCALE_E8M0", "AR_FMT_BF16", "AR_FMT_F32", "AR_NORM_MAX_COLS",
    "ar_rope_kv", "ar_attn_decode", "ar_attn", "ar_attn_paged", "ar_attn_bwd", "attn_decode_workspace",
    "attn_bwd_workspace", "kv_cache_empty", "rope_table",
    "AR_FMT_E4M3", "AR_ATTN_MAX_DIM", "AR_ROPE_PAIRS", "AR_ROPE_INVERSE",
]

AR_OK = 0
AR_ERR_INVALID = -1
AR_ERR_ALIGN = -2
AR_ERR_ALIAS = -3
AR_ERR_UNSUPPORTED = -4
AR_ERR_HIP = -5
AR_ERR_SIZE = -6
AR_STATIC_SCRATCH_ELEMS = 16777216
AR_MAX_RANKS = 8
AR_VARIANT_ONESHOT = 0
AR_VARIANT_2STAGE = 1
AR_UBATCH_BOUNDED = 256
AR_RD_STAGED = 1
AR_RD_FP32_CARRY = 2
AR_KERNEL_ONESHOT = 0
AR_KERNEL_2STAGE = 1
AR_KERNEL_UBATCH = 2
AR_KERNEL_RS = 3
AR_KERNEL_AG = 4
AR_KERNEL_PACK = 5
AR_KERNEL_UNPACK = 6
AR_KERNEL_RD = 7
AR_KERNEL_RDSTEP = 8
AR_KERNEL_UNPACK_WAIT = 9
AR_KERNEL_UBATCH_FLAGS = 10
AR_KERNEL_QUANT_FP8 = 11
AR_KERNEL_REDUCE_FP8 = 12
AR_KERNEL_REDUCE_FP8_ALL = 13
AR_KERNEL_ONESHOT_SMALL = 14
AR_KERNEL_2STAGE_SMALL = 15
AR_KERNEL_RD_SMALL = 16
AR_KERNEL_RDSTEP_SMALL = 17
AR_KERNEL_PACK_SMALL = 18
AR_KERNEL_UNPACK_SMALL = 19
AR_KERNEL_UBATCH_BOUNDED = 20
AR_KERNEL_2STAGE_INPLACE_SMALL = 21
AR_SMALL_ELEMS = 2097152
FP8_BLOCK = 32                  # elements per power-of-two scale
AR_BLOCK = 128                  # columns per scale of an fp8 matrix
AR_SCALE_F32 = 0
AR_SCALE_E8M0 = 1
AR_FMT_BF16 = 0
AR_FMT_F32 = 1
AR_NORM_MAX_COLS = 65536
AR_FMT_E4M3 = 2
AR_ATTN_MAX_DIM = 128
AR_ROPE_PAIRS = 1
AR_ROPE_INVERSE = 2

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libarcore.so")
_lib = None

_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_u32 = ctypes.c_uint32


class _Fp8Matrix(ctypes.Structure):
    """ar_fp8_matrix"""
    _fields_ = [("codes", _vp), ("ld", _sz), ("scales", _vp), ("scale_rs", _sz), ("scale_cs", _sz),
                ("scale_fmt", ctypes.c_int), ("block_rows", ctypes.c_int)]


class _Heads(ctypes.Structure):
    """ar_heads"""
    _fields_ = [("data", _vp), ("token_stride", _sz), ("head_stride", _sz)]


class _KVCache(ctypes.Structure):
    """ar_kv_cache"""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp)] + [
        (n, _sz) for n in ("pages", "page_size", "heads", "dim", "page_stride", "token_stride", "head_stride",
                           "scale_page_stride", "scale_token_stride", "scale_head_stride")] + [("fmt", ctypes.c_int)]


class ARError(RuntimeError):
    """A nonzero status from the C-ABI."""

    def __init__(self, code: int, func: str):
        self.code = code
        super().__init__(f"{func}: {ar_status_str(code)} ({code})")


def lib():
    """Load libarcore.so from this package directory (raises if absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError(f"{lib_path} is not built; run __graft_entry__.build() "
                              "(hipcc --offload-arch=gfx950)")
        L = ctypes.CDLL(lib_path)
        L.ar_status_str.restype = ctypes.c_char_p
        L.ar_status_str.argtypes = [ctypes.c_int]
        L.ar_version.restype = ctypes.c_int
        L.ar_version.argtypes = []
        L.ar_reduce_oneshot.restype = ctypes.c_int
        L.ar_reduce_oneshot.argtypes = [ctypes.POINTER(_vp), ctypes.c_int, _vp, _sz, _vp]
        L.ar_reduce_2stage.restype = ctypes.c_int
        L.ar_reduce_2stage.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, _sz,
                                       _vp, _vp]
        L.ar_reduce_2stage_static.restype = ctypes.c_int
        L.ar_reduce_2stage_static.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, _sz, _vp]
        L.ar_pack_fused.restype = ctypes.c_int
        L.ar_pack_fused.argtypes = [_vp, _vp, _sz, _u32, _vp]
        L.ar_unpack_fused.restype = ctypes.c_int
        L.ar_unpack_fused.argtypes = [_vp, _vp, _sz, _u32, _vp, _vp]
        L.ar_unpack_fused_wait.restype = ctypes.c_int
        L.ar_unpack_fused_wait.argtypes = [_vp, _vp, _sz, _u32, _u32, _vp, _vp]
        L.ar_rd_schedule.restype = ctypes.c_int
        L.ar_rd_schedule.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, _sz,
                                     _u32, _vp, ctypes.c_int, _vp, _vp]
        L.ar_reduce_ubatch.restype = ctypes.c_int
        L.ar_reduce_ubatch.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, _sz,
                                       _sz, ctypes.c_int, ctypes.POINTER(_sz), _sz, ctypes.c_int,
                                       ctypes.POINTER(_vp)]
        L.ar_reduce_ubatch_flags.restype = ctypes.c_int
        L.ar_reduce_ubatch_flags.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, _sz,
                                             _sz, ctypes.c_int, ctypes.POINTER(_sz), _sz, ctypes.c_int,
                                             ctypes.POINTER(_vp), _vp, _vp, _sz, _u32]
        L.ar_err_init.restype = ctypes.c_int
        L.ar_err_init.argtypes = [_vp, _vp]
        L.ar_quantize_fp8.restype = ctypes.c_int
        L.ar_quantize_fp8.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                      ctypes.c_int, _sz, _vp]
        L.ar_reduce_fp8.restype = ctypes.c_int
        L.ar_reduce_fp8.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int,
                                    ctypes.POINTER(_vp), ctypes.c_int, _sz, _vp]
        mp, f32 = ctypes.POINTER(_Fp8Matrix), ctypes.c_float
        L.ar_reduce_norm.restype = ctypes.c_int
        L.ar_reduce_norm.argtypes = [ctypes.POINTER(_vp), ctypes.c_int, _vp, _vp, ctypes.c_int, _sz, _sz, f32, _vp,
                                     _vp, mp, _vp]
        L.ar_norm_bwd_workspace.restype = _sz
        L.ar_norm_bwd_workspace.argtypes = [_sz, _sz]
        L.ar_norm_bwd.restype = ctypes.c_int
        L.ar_norm_bwd.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _sz, _sz, f32, _vp, _vp, _vp, _sz, _vp]
        L.ar_quantize_block.restype = ctypes.c_int
        L.ar_quantize_block.argtypes = [_vp, _sz, _sz, _sz, mp, ctypes.c_int, _vp]
        L.ar_gemm_fp8_workspace.restype = _sz
        L.ar_gemm_fp8_workspace.argtypes = [_sz, _sz, _sz, ctypes.c_int]
        L.ar_gemm_fp8.restype = ctypes.c_int
        L.ar_gemm_fp8.argtypes = [mp, mp, ctypes.POINTER(_vp), ctypes.c_int, _sz, _sz, _sz, _sz, ctypes.c_int, _vp,
                                  _sz, _vp]
        hp, cp = ctypes.POINTER(_Heads), ctypes.POINTER(_KVCache)
        tail = [_sz, _sz]                       # window, sinks
        res = [hp, _vp, _sz, _sz]               # out, lse and its strides
        L.ar_rope_kv.restype = ctypes.c_int
        L.ar_rope_kv.argtypes = [hp, hp, hp, _sz, _sz, _sz, _sz, _vp, _sz, _sz, _vp, hp, hp, cp, _vp, ctypes.c_int, _vp]
        L.ar_attn_decode_workspace.restype = _sz
        L.ar_attn_decode_workspace.argtypes = [_sz] * 4
        L.ar_attn_decode.restype = ctypes.c_int
        L.ar_attn_decode.argtypes = [hp, cp, _vp, _sz, _sz, _vp, _sz, _sz, f32, *tail, *res, _vp, _sz, _vp]
        L.ar_attn.restype = ctypes.c_int
        L.ar_attn.argtypes = [hp, hp, hp, _vp, _vp] + [_sz] * 6 + [f32, *tail, *res, _vp]
        L.ar_attn_paged.restype = ctypes.c_int
        L.ar_attn_paged.argtypes = [hp, cp, _vp, _sz, _sz, _vp, _vp, _sz, _sz, _sz, f32, *tail, *res, _vp]
        L.ar_attn_bwd_workspace.restype = _sz
        L.ar_attn_bwd_workspace.argtypes = [_sz] * 8
        L.ar_attn_bwd.restype = ctypes.c_int
        L.ar_attn_bwd.argtypes = [hp, hp, hp, hp, _vp, _sz, _sz, hp, _vp, _vp] + [_sz] * 6 + [f32, *tail, hp, hp, hp, _vp,
                                                                                             _sz, _vp]
        L.ar_set_launch_shape.restype = ctypes.c_int
        L.ar_set_launch_shape.argtypes = [ctypes.c_int] * 6
        ip = ctypes.POINTER(ctypes.c_int)
        L.ar_get_launch_shape.restype = ctypes.c_int
        L.ar_get_launch_shape.argtypes = [ctypes.c_int, ip, ip, ip, ip, ip]
        _lib = L
    return _lib


def ar_status_str(code: int) -> str:
    return lib().ar_status_str(int(code)).decode()


def ar_version() -> int:
    return int(lib().ar_version())


# ---------------------------------------------------------------- marshalling

def _check(rc: int, func: str) -> None:
    if rc != AR_OK:
        raise ARError(rc, func)


_tls = threading.local()


def _call(name: str, *cargs) -> None:
    """Make one device call of the library with marshalled arguments, or,
    inside prepare(), record it instead of making it."""
    fn = getattr(lib(), name)
    slot = getattr(_tls, "capture", None)
    if slot is not None:
        slot.append((fn, name, cargs))
        return
    _check(fn(*cargs), name)


class Prepared:
    """One device call with its arguments checked and marshalled once.

    Calling it makes the same C-ABI call as the wrapper it was prepared from,
    with the same device pointers, sizes and stream, and raises ARError on a
    nonzero status.  It holds references to the tensors it was prepared
    with, so their storage stays allocated while the handle lives; their
    contents may change between calls (that is the point), their storage
    must not be replaced (``set_``, ``resize_``).  The stream is the one
    named at prepare time, or the current stream then if none was named.
    """

    __slots__ = ("_fn", "_name", "_args", "_refs")

    def __init__(self, fn, name: str, cargs: tuple, refs: tuple):
        if len(cargs) != len(fn.argtypes):
            raise TypeError(f"{name}: {len(cargs)} arguments for {len(fn.argtypes)} parameters")
        # plain ints become instances of the declared C types now, which
        # ctypes then passes through as they are (about 0.1 us a call)
        conv = tuple(t(a) if isinstance(a, int) else a for a, t in zip(cargs, fn.argtypes))
        self._fn, self._name, self._args, self._refs = fn, name, conv, refs

    @property
    def name(self) -> str:
        return self._name

    def __call__(self) -> None:
        rc = self._fn(*self._args)
        if rc != AR_OK:
            raise ARError(rc, self._name)

    def __repr__(self) -> str:
        return f"<Prepared {self._name}>"


def prepare(func, *args, **kwargs) -> Prepared:
    """Check and marshal the arguments of one device call once.

    ``prepare(ar_reduce_2stage, ins, outs)`` validates ``ins`` and ``outs``
    exactly as ``ar_reduce_2stage(ins, outs)`` would (raising the same
    errors), queues nothing, and returns a Prepared handle whose call queues
    that work.  For loops that pass the same buffers on every step (a decode
    step's all-reduce): a wrapper call spends about 0.45 us per tensor in
    checks and pointer lookups, a prepared call none.  ``func`` is one of the
    device calls of this module."""
    if func not in _PREPARABLE and func not in _PREPARABLE_BLOCK and func not in _PREPARABLE_ATTN:
        raise ValueError(f"prepare() takes a device call of this module, not {func!r}")
    slot = []
    _tls.capture = slot
    try:
        func(*args, **kwargs)
    finally:
        _tls.capture = None
    (fn, name, cargs), = slot
    return Prepared(fn, name, cargs, (args, kwargs))


def _dev_ptr(t, elem_size: int, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.element_size() != elem_size:
        raise ValueError(f"{name} must have {elem_size}-byte elements")
    return t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr_array(ptrs):
    arr = (_vp * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr


def _bufs(ts, elem_size: int, name: str, count: int | None = None):
    ptrs = []
    for i, t in enumerate(ts):
        if t is None:
            ptrs.append(None)
            continue
        if count is not None and t.numel() < count:
            raise ValueError(f"{name}[{i}] holds {t.numel()} elements, {count} needed")
        ptrs.append(_dev_ptr(t, elem_size, f"{name}[{i}]"))
    return ptrs


def ar_reduce_oneshot(ins: Sequence, out, n: int | None = None, stream=None) -> None:
    """out[:n] = sum of ins[p][:n] (binary32 accumulation in rank order, one bf16 rounding)."""
    n = ins[0].numel() if n is None else int(n)
    ip = _bufs(ins, 2, "ins", n)
    (op,) = _bufs([out], 2, "out", n)
    _call("ar_reduce_oneshot", _ptr_array(ip), len(ip), op, n, _stream(stream))


def ar_reduce_2stage(ins: Sequence, outs: Sequence, scratch=None, n: int | None = None,
                     stream=None) -> None:
    """Every outs[r][:n] = the one-shot sum; scratch given -> staged RS/AG.
    outs may be ins itself (in place: each rank's result in its own buffer)."""
    n = ins[0].numel() if n is None else int(n)
    ip = _bufs(ins, 2, "ins", n)
    op = _bufs(outs, 2, "outs", n)
    if len(op) != len(ip):
        raise ValueError("need one output per rank")
    sp = None if scratch is None else _bufs([scratch], 2, "scratch", n)[0]
    _call("ar_reduce_2stage", _ptr_array(ip), _ptr_array(op), len(ip), n, sp, _stream(stream))


def ar_reduce_2stage_static(ins: Sequence, outs: Sequence, n: int | None = None, stream=None) -> None:
    """The staged two-stage reduce through the library's static scratch (no
    allocation, no workspace argument); n <= AR_STATIC_SCRATCH_ELEMS."""
    n = ins[0].numel() if n is None else int(n)
    ip = _bufs(ins, 2, "ins", n)
    op = _bufs(outs, 2, "outs", n)
    if len(op) != len(ip):
        raise ValueError("need one output per rank")
    _call("ar_reduce_2stage_static", _ptr_array(ip), _ptr_array(op), len(ip), n, _stream(stream))


def ar_pack_fused(x, words, seq: int, n: int | None = None, stream=None) -> None:
    n = x.numel() if n is None else int(n)
    (xp,) = _bufs([x], 2, "x", n)
    (wp,) = _bufs([words], 8, "words", n // 2)
    _call("ar_pack_fused", xp, wp, n, int(seq) & 0xFFFFFFFF, _stream(stream))


def ar_unpack_fused(words, x, expected_seq: int, d_err, n: int | None = None, stream=None) -> None:
    n = x.numel() if n is None else int(n)
    (wp,) = _bufs([words], 8, "words", n // 2)
    (xp,) = _bufs([x], 2, "x", n)
    (ep,) = _bufs([d_err], 8, "d_err", 2)
    _call("ar_unpack_fused", wp, xp, n, int(expected_seq) & 0xFFFFFFFF, ep, _stream(stream))


def ar_unpack_fused_wait(words, x, expected_seq: int, d_err, max_spins: int = 1 << 20,
                         n: int | None = None, stream=None) -> None:
    """Unpack, waiting (at most max_spins polls per wavefront) for a
    concurrent producer to write payloads carrying expected_seq."""
    n = x.numel() if n is None else int(n)
    (wp,) = _bufs([words], 8, "words", n // 2)
    (xp,) = _bufs([x], 2, "x", n)
    (ep,) = _bufs([d_err], 8, "d_err", 2)
    _call("ar_unpack_fused_wait", wp, xp, n, int(expected_seq) & 0xFFFFFFFF, int(max_spins), ep,
          _stream(stream))


def rd_mailbox_words(P: int, n: int) -> int:
    """Mailbox size in payload words for ar_rd_schedule(..., AR_RD_STAGED)."""
    steps = {2: 1, 4: 2, 8: 3}[P]
    W = n // 2
    return P * (steps - 1) * (W + (W & 1))


def ar_rd_schedule(in_words: Sequence, out_words: Sequence, seq0: int, d_err, mailbox=None,
                   flags: int = 0, n: int | None = None, stream=None) -> None:
    n = 2 * in_words[0].numel() if n is None else int(n)
    ip = _bufs(in_words, 8, "in_words", n // 2)
    op = _bufs(out_words, 8, "out_words", n // 2)
    if len(op) != len(ip):
        raise ValueError("need one output payload per rank")
    mp = None
    if mailbox is not None:
        (mp,) = _bufs([mailbox], 8, "mailbox", rd_mailbox_words(len(ip), n) if len(ip) in (2, 4, 8) else 0)
    (ep,) = _bufs([d_err], 8, "d_err", 2)
    _call("ar_rd_schedule", _ptr_array(ip), _ptr_array(op), len(ip), n, int(seq0) & 0xFFFFFFFF,
          mp, int(flags), ep, _stream(stream))


def ar_reduce_ubatch(ins: Sequence, outs: Sequence, rows: int, hidden: int, n_ubatch: int = 2,
                     ubatch_rows: Sequence[int] | None = None, chunk_bytes: int = 1 << 20,
                     variant: int = AR_VARIANT_2STAGE, streams: Sequence | None = None) -> None:
    n = int(rows) * int(hidden)
    ip = _bufs(ins, 2, "ins", n)
    op = _bufs(outs, 2, "outs", n)
    if streams is None:
        streams = [None] * n_ubatch
    if len(streams) != n_ubatch:
        raise ValueError("need one stream per ubatch")
    sp = _ptr_array([_stream(s) for s in streams])
    ub = None
    if ubatch_rows is not None:
        if len(ubatch_rows) != n_ubatch:
            raise ValueError("need one row count per ubatch")
        ub = (_sz * n_ubatch)(*[int(r) for r in ubatch_rows])
    _call("ar_reduce_ubatch", _ptr_array(ip), _ptr_array(op), len(ip), int(rows), int(hidden),
          int(n_ubatch), ub, int(chunk_bytes), int(variant), sp)


def ubatch_chunk_count(rows: int, hidden: int, n_ubatch: int = 2, ubatch_rows=None,
                       chunk_bytes: int = 1 << 20) -> int:
    """Total chunks of a ubatch reduce (size of the flag arrays)."""
    if ubatch_rows is None:
        ubatch_rows = [rows // n_ubatch] * (n_ubatch - 1)
        ubatch_rows.append(rows - sum(ubatch_rows))
    ce = chunk_bytes // 2
    return sum((int(r) * hidden + ce - 1) // ce for r in ubatch_rows)


def ar_reduce_ubatch_flags(ins: Sequence, outs: Sequence, rows: int, hidden: int, chunk_done,
                           chunk_tiles, epoch: int, n_ubatch: int = 2,
                           ubatch_rows: Sequence[int] | None = None, chunk_bytes: int = 1 << 20,
                           variant: int = AR_VARIANT_2STAGE, streams: Sequence | None = None) -> None:
    """ar_reduce_ubatch that also publishes done[chunk] = epoch per chunk."""
    n = int(rows) * int(hidden)
    ip = _bufs(ins, 2, "ins", n)
    op = _bufs(outs, 2, "outs", n)
    if streams is None:
        streams = [None] * n_ubatch
    if len(streams) != n_ubatch:
        raise ValueError("need one stream per ubatch")
    sp = _ptr_array([_stream(s) for s in streams])
    ub = None
    if ubatch_rows is not None:
        if len(ubatch_rows) != n_ubatch:
            raise ValueError("need one row count per ubatch")
        ub = (_sz * n_ubatch)(*[int(r) for r in ubatch_rows])
    (dp,) = _bufs([chunk_done], 4, "chunk_done")
    (tp,) = _bufs([chunk_tiles], 4, "chunk_tiles")
    nf = min(chunk_done.numel(), chunk_tiles.numel())
    _call("ar_reduce_ubatch_flags", _ptr_array(ip), _ptr_array(op), len(ip), int(rows), int(hidden),
          int(n_ubatch), ub, int(chunk_bytes), int(variant), sp, dp, tp, nf, int(epoch) & 0xFFFFFFFF)


def fp8_scale_count(n: int) -> int:
    """Scale bytes per rank for n elements: one per block of 32."""
    return -(-int(n) // FP8_BLOCK)


def ar_quantize_fp8(xs: Sequence, codes: Sequence, scales: Sequence, n: int | None = None,
                    stream=None) -> None:
    """Quantise P bf16 buffers to E4M3 codes (uint8[n]) and per-32-element
    power-of-two scales (uint8[ceil(n/32)], exponent + 127), one launch."""
    n = xs[0].numel() if n is None else int(n)
    xp = _bufs(xs, 2, "xs", n)
    cp = _bufs(codes, 1, "codes", n)
    sp = _bufs(scales, 1, "scales", fp8_scale_count(n))
    if not (len(xp) == len(cp) == len(sp)):
        raise ValueError("need one code and one scale buffer per input")
    _call("ar_quantize_fp8", _ptr_array(xp), _ptr_array(cp), _ptr_array(sp), len(xp), n, _stream(stream))


def ar_reduce_fp8(codes: Sequence, scales: Sequence, outs: Sequence, n: int | None = None,
                  stream=None) -> None:
    """outs[r][:n] = rank-order binary32 sum of the dequantised contributions,
    rounded to bf16; len(outs) is 1 (one share) or P (all-reduce)."""
    n = codes[0].numel() if n is None else int(n)
    cp = _bufs(codes, 1, "codes", n)
    sp = _bufs(scales, 1, "scales", fp8_scale_count(n))
    op = _bufs(outs, 2, "outs", n)
    if len(cp) != len(sp):
        raise ValueError("need one scale buffer per code buffer")
    _call("ar_reduce_fp8", _ptr_array(cp), _ptr_array(sp), len(cp), _ptr_array(op), len(op), n,
          _stream(stream))


# ------------------------------------------- norm, block quantiser, fp8 product

# Element types by what the kernels read them as: the type itself, or its bit
# patterns in whole numbers.
_BF16 = ("bfloat16", "int16", "uint16")
_F32 = ("float32",)
_E4M3 = ("float8_e4m3fn", "uint8", "int8")
_E8M0 = ("float8_e8m0fnu", "uint8", "int8")


def _typed(t, kinds, name: str) -> None:
    """Refuses a tensor of another element type, which its bytes would be
    misread as."""
    dtype = getattr(t, "dtype", None)
    if dtype is not None and str(dtype).rpartition(".")[2] not in kinds:
        raise ValueError(f"{name} must have elements of type {' or '.join(kinds)}, not {dtype}")


def _mat(t, elem_sizes, name: str, shape=None):
    """(pointer, row stride in elements) of a 2-D device tensor whose rows
    are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must have shape {'(rows, cols)' if shape is None else tuple(shape)}, "
                         f"not {tuple(t.shape)}")
    if t.element_size() not in elem_sizes:
        raise ValueError(f"{name} must have {' or '.join(map(str, elem_sizes))}-byte elements")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), (t.stride(0) if rows > 1 else cols)


def _rows_of(t, name: str, shape):
    """Pointer of a contiguous bf16 matrix of that shape."""
    ptr = _dev_ptr(t, 2, name)
    _typed(t, _BF16, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return ptr


def _fp8_matrix(codes, scales, shape, block_rows: int, name: str) -> _Fp8Matrix:
    rows, cols = shape
    ptr, ld = _mat(codes, (1,), f"{name} codes", shape)
    _typed(codes, _E4M3, f"{name} codes")
    if rows <= 1:
        ld = -(-cols // 16) * 16
    want = (-(-rows // block_rows), -(-cols // AR_BLOCK))
    if not scales.is_cuda:
        raise ValueError(f"{name} scales must be a device tensor")
    if tuple(scales.shape) != want:
        raise ValueError(f"{name} scales must have shape {want}, not {tuple(scales.shape)}")
    if scales.element_size() == 4 and scales.is_floating_point():
        fmt = AR_SCALE_F32
    elif scales.element_size() == 1:
        fmt = AR_SCALE_E8M0
    else:
        raise ValueError(f"{name} scales must be binary32 or power-of-two bytes")
    _typed(scales, _F32 if fmt == AR_SCALE_F32 else _E8M0, f"{name} scales")
    # the stride of an axis of one block says nothing
    rs = scales.stride(0) if want[0] > 1 else 0
    cs = scales.stride(1) if want[1] > 1 else 0
    return _Fp8Matrix(ptr, ld, scales.data_ptr(), rs, cs, fmt, block_rows)


def _gain(weight, cols: int):
    if weight is None:
        return None, AR_FMT_BF16
    if weight.numel() != cols:
        raise ValueError(f"weight holds {weight.numel()} elements, {cols} needed")
    es = weight.element_size()
    if es not in (2, 4):
        raise ValueError("weight must be bf16 or binary32")
    _typed(weight, _F32 if es == 4 else _BF16, "weight")
    return _dev_ptr(weight, es, "weight"), AR_FMT_F32 if es == 4 else AR_FMT_BF16


def fp8_codes_empty(rows: int, cols: int, device, dtype=None):
    """An uninitialised [rows, cols] code matrix whose rows start on 16-byte
    boundaries (uint8, or `dtype`, e.g. torch.float8_e4m3fn)."""
    import torch
    ld = -(-int(cols) // 16) * 16
    return torch.empty(int(rows), ld, dtype=dtype or torch.uint8, device=device)[:, :int(cols)]


def fp8_scales_empty(rows: int, cols: int, device, block_rows: int = 1, e8m0: bool = False):
    """Uninitialised scales of a [rows, cols] matrix, shape [ceil(rows /
    block_rows), ceil(cols / 128)], binary32 or (e8m0) bytes; stored block
    column by block column, so that ar_gemm_fp8 reads consecutive rows'
    scales from consecutive addresses."""
    import torch
    return torch.empty(-(-int(cols) // AR_BLOCK), -(-int(rows) // block_rows), device=device,
                       dtype=torch.uint8 if e8m0 else torch.float32).t()


def ar_reduce_norm(ins: Sequence, weight=None, residual=None, res_out=None, y=None, codes=None, scales=None,
                   eps: float = 1e-6, stream=None) -> None:
    """h = sum of ins[p] (+ residual), res_out = bf16(h), y = h / rms(h) *
    weight as bf16 (`y`) and / or E4M3 with a scale for each 128 columns
    (`codes`, `scales`).  All of ins, residual, res_out and y are contiguous
    [rows, cols] matrices; codes may have padded rows (a stride that is a
    multiple of 16), scales any strides."""
    if ins[0].dim() != 2:
        raise ValueError("ins must be [rows, cols] matrices")
    rows, cols = shape = tuple(ins[0].shape)
    ip = [_rows_of(t, f"ins[{i}]", shape) for i, t in enumerate(ins)]
    rp = None if residual is None else _rows_of(residual, "residual", shape)
    op = None if res_out is None else _rows_of(res_out, "res_out", shape)
    yp = None if y is None else _rows_of(y, "y", shape)
    wp, wf = _gain(weight, cols)
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales come together")
    q = None if codes is None else ctypes.pointer(_fp8_matrix(codes, scales, shape, 1, "output"))
    _call("ar_reduce_norm", _ptr_array(ip), len(ip), rp, wp, wf, rows, cols, ctypes.c_float(eps), op, yp, q,
          _stream(stream))


def norm_bwd_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that ar_norm_bwd needs for dweight."""
    return int(lib().ar_norm_bwd_workspace(int(rows), int(cols)))


def ar_norm_bwd(dy, h, weight=None, dx=None, dres=None, dweight=None, workspace=None, eps: float = 1e-6,
                stream=None) -> None:
    """Gradient of ar_reduce_norm's norm: dx (of h: of every contribution and
    of the residual; dres is the gradient that reached res_out) and dweight
    (binary32).  dweight needs norm_bwd_workspace(rows, cols) bytes."""
    if h.dim() != 2:
        raise ValueError("h must be a [rows, cols] matrix")
    rows, cols = shape = tuple(h.shape)
    yp, hp = _rows_of(dy, "dy", shape), _rows_of(h, "h", shape)
    rp = None if dres is None else _rows_of(dres, "dres", shape)
    xp = None if dx is None else _rows_of(dx, "dx", shape)
    wp, wf = _gain(weight, cols)
    dp = None
    if dweight is not None:
        if dweight.numel() != cols:
            raise ValueError(f"dweight holds {dweight.numel()} elements, {cols} needed")
        dp = _dev_ptr(dweight, 4, "dweight")
        _typed(dweight, _F32, "dweight")
    sp, sb = _workspace(workspace)
    _call("ar_norm_bwd", yp, hp, wp, wf, rp, rows, cols, ctypes.c_float(eps), xp, dp, sp, sb, _stream(stream))


def _workspace(t):
    if t is None or t.numel() == 0:
        return None, 0
    return _dev_ptr(t, t.element_size(), "workspace"), t.numel() * t.element_size()


def ar_quantize_block(x, codes, scales, block_rows: int = 1, transpose: bool = False, stream=None) -> None:
    """Quantise a bf16 matrix (rows contiguous, any row stride) to E4M3 codes
    with a scale for each block of block_rows (1 or 128) x 128; transpose:
    codes and scales are those of x transposed."""
    xp, ldx = _mat(x, (2,), "x")
    _typed(x, _BF16, "x")
    rows, cols = x.shape
    q = _fp8_matrix(codes, scales, (cols, rows) if transpose else (rows, cols), int(block_rows), "output")
    _call("ar_quantize_block", xp, ldx, rows, cols, ctypes.pointer(q), int(bool(transpose)), _stream(stream))


def gemm_fp8_workspace(M: int, N: int, K: int, G: int = 1) -> int:
    """Bytes of workspace with which ar_gemm_fp8 may split a product along K
    (zero-initialised once by the caller; 0: none is used)."""
    return int(lib().ar_gemm_fp8_workspace(int(M), int(N), int(K), int(G)))


def ar_gemm_fp8(a_codes: Sequence, a_scales: Sequence, b_codes: Sequence, b_scales: Sequence, outs: Sequence,
                b_block_rows: int = 128, workspace=None, stream=None) -> None:
    """outs[g] = a[g] b[g]^T for len(outs) fp8 problems of one shape: a [M, K]
    with a scale for each 1 x 128 block, b [N, K] with one for each
    b_block_rows x 128, outs [M, N] bf16 or binary32 by their element size."""
    G = len(outs)
    if not (G == len(a_codes) == len(a_scales) == len(b_codes) == len(b_scales)) or G == 0:
        raise ValueError("need one matrix and one scale matrix of a and of b, and one output, per problem")
    if a_codes[0].dim() != 2 or b_codes[0].dim() != 2:
        raise ValueError("a and b must be matrices")
    (M, K), N = tuple(a_codes[0].shape), int(b_codes[0].shape[0])
    am = (_Fp8Matrix * G)(*[_fp8_matrix(c, s, (M, K), 1, f"a[{i}]") for i, (c, s) in enumerate(zip(a_codes, a_scales))])
    bm = (_Fp8Matrix * G)(*[_fp8_matrix(c, s, (N, K), int(b_block_rows), f"b[{i}]")
                            for i, (c, s) in enumerate(zip(b_codes, b_scales))])
    es = outs[0].element_size()
    cp = []
    for i, t in enumerate(outs):
        ptr, ld = _mat(t, (2, 4), f"outs[{i}]", (M, N))
        if t.element_size() != es or ld != _mat(outs[0], (2, 4), "outs[0]")[1]:
            raise ValueError("outs must share one element size and one row stride")
        _typed(t, _F32 if es == 4 else _BF16, f"outs[{i}]")
        cp.append(ptr)
    sp, sb = _workspace(workspace)
    _call("ar_gemm_fp8", am, bm, _ptr_array(cp), G, M, N, K, ld, AR_FMT_F32 if es == 4 else AR_FMT_BF16, sp, sb,
          _stream(stream))


# ------------------------------------------------------------------ attention

_I32 = ("int32",)
_I64 = ("int64",)


def _here(tensors) -> None:
    """Refuses tensors that are not all on the current device, on which the
    call's work is queued."""
    import torch
    where = {t.device for t in tensors if t is not None and getattr(t, "device", None) is not None}
    if len(where) > 1 or (where and next(iter(where)).index != torch.cuda.current_device()):
        raise ValueError("all tensors of a call must be on the current device")


def _heads(t, name: str, shape=None):
    """ar_heads of a [tokens, heads, dim] tensor whose dim is contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 3 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must have shape {'(tokens, heads, dim)' if shape is None else tuple(shape)}, "
                         f"not {tuple(t.shape)}")
    _typed(t, _BF16, name)
    if t.element_size() != 2:
        raise ValueError(f"{name} must have 2-byte elements")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous heads")
    # the stride of an axis of one element says nothing
    return ctypes.pointer(_Heads(t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0))


def _ints(t, kinds, name: str, count: int):
    if t.dim() != 1 or t.shape[0] != count:
        raise ValueError(f"{name} must have shape ({count},), not {tuple(t.shape)}")
    _typed(t, kinds, name)
    return _dev_ptr(t, 8 if kinds is _I64 else 4, name)


def _kv_cache(cache):
    """ar_kv_cache of (keys, values) or (keys, values, their scales)."""
    if len(cache) not in (2, 4):
        raise ValueError("a cache is (k, v), or (k, v, k_scales, v_scales) of E4M3 codes")
    k, v = cache[:2]
    small = len(cache) == 4
    for t, name in ((k, "cache keys"), (v, "cache values")):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if t.dim() != 4 or tuple(t.shape) != tuple(k.shape):
            raise ValueError(f"{name} must have shape (pages, page_size, heads, dim), both the same")
        _typed(t, _E4M3 if small else _BF16, name)
        if t.element_size() != (1 if small else 2):
            raise ValueError(f"{name} must have {1 if small else 2}-byte elements")
        if t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError(f"{name} must have contiguous heads")
        if _steps(t, 3) != _steps(k, 3):
            raise ValueError("cache keys and values must have the same strides")
    steps, ptrs = _steps(k, 3), [None, None]
    scale_steps = (0, 0, 0)
    if small:
        scale_steps = _steps(cache[2], 3)
        for i, (t, name) in enumerate(zip(cache[2:], ("cache k_scales", "cache v_scales"))):
            if not t.is_cuda:
                raise ValueError(f"{name} must be a device tensor")
            if tuple(t.shape) != tuple(k.shape[:3]):
                raise ValueError(f"{name} must have shape {tuple(k.shape[:3])}, not {tuple(t.shape)}")
            _typed(t, _F32, name)
            if _steps(t, 3) != scale_steps:
                raise ValueError("cache scales must have the same strides")
            ptrs[i] = t.data_ptr()
    return ctypes.pointer(_KVCache(k.data_ptr(), v.data_ptr(), *ptrs, *k.shape, *steps, *scale_steps,
                                   AR_FMT_E4M3 if small else AR_FMT_BF16))


def _steps(t, n: int) -> tuple:
    """The first n strides; 0 of an axis of one element."""
    return tuple(t.stride(i) if t.shape[i] > 1 else 0 for i in range(n))


def _lse(lse, shape):
    if lse is None:
        return None, 0, 0
    if not lse.is_cuda:
        raise ValueError("lse must be a device tensor")
    if tuple(lse.shape) != tuple(shape):
        raise ValueError(f"lse must have shape {tuple(shape)}, not {tuple(lse.shape)}")
    _typed(lse, _F32, "lse")
    return (lse.data_ptr(), *_steps(lse, 2))


def _mask(scale, dim: int, window: int, sinks: int):
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    return ctypes.c_float(dim ** -0.5 if scale is None else scale), int(window), int(sinks)


def kv_cache_empty(pages: int, page_size: int, heads: int, dim: int, device, e4m3: bool = False):
    """An uninitialised cache: (k, v) of shape [pages, page_size, heads, dim]
    in bf16, or (k, v, k_scales, v_scales) with E4M3 codes."""
    import torch
    shape = (int(pages), int(page_size), int(heads), int(dim))
    kv = tuple(torch.empty(shape, device=device, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2))
    return kv + tuple(torch.empty(shape[:3], device=device, dtype=torch.float32) for _ in range(2)) if e4m3 else kv


def rope_table(positions: int, rot: int, theta: float = 10000.0, device="cuda"):
    """cos_sin of ar_rope_kv for positions 0 ... positions - 1: the angle of
    pair i is position * theta^(-2 i / rot), formed in 64 bits."""
    import torch
    freq = float(theta) ** (-torch.arange(0, int(rot), 2, device=device, dtype=torch.float64) / int(rot))
    angle = torch.arange(int(positions), device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def ar_rope_kv(q, k, v, cos_sin, positions, q_out=None, k_out=None, cache=None, slots=None, pairs: bool = False,
               inverse: bool = False, stream=None) -> None:
    """Rotates q and k [tokens, heads, dim] by their positions (int32) into
    q_out and k_out (each may be its input) and puts rotated keys and v into
    the cache's slots (int64, page * page_size + place; -1: nowhere).
    cos_sin [positions, rot] binary32: rot / 2 cosines, then the sines
    (rope_table).  pairs: neighbours are rotated together, not elements half
    of rot apart.  inverse: the rotation back, which is the gradient.  q, or
    k and v, may be None."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("need q or k")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if (cache is None) != (slots is None):
        raise ValueError("cache and slots come together")
    if some.dim() != 3:
        raise ValueError("q and k must have shape (tokens, heads, dim)")
    tokens, _, dim = some.shape
    hq = 0 if q is None else int(q.shape[1])
    hkv = 0 if k is None else int(k.shape[1])
    qp = None if q is None else _heads(q, "q", (tokens, hq, dim))
    qo = None if q is None else _heads(q_out, "q_out", (tokens, hq, dim))
    kp = None if k is None else _heads(k, "k", (tokens, hkv, dim))
    vp = None if v is None else _heads(v, "v", (tokens, hkv, dim))
    ko = None if k_out is None else _heads(k_out, "k_out", (tokens, hkv, dim))
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must have shape (positions, rot)")
    rows, rot = cos_sin.shape
    _typed(cos_sin, _F32, "cos_sin")
    tp = _dev_ptr(cos_sin, 4, "cos_sin")
    pp = _ints(positions, _I32, "positions", tokens)
    cp = sp = None
    if cache is not None:
        cp, sp = _kv_cache(cache), _ints(slots, _I64, "slots", tokens)
    _here([q, k, v, cos_sin, positions, q_out, k_out, slots, *(cache or ())])
    _call("ar_rope_kv", qp, kp, vp, tokens, hq, hkv, dim, tp, rows, rot, pp, qo, ko, cp, sp,
          (AR_ROPE_PAIRS if pairs else 0) | (AR_ROPE_INVERSE if inverse else 0), _stream(stream))


def attn_decode_workspace(seqs: int, hq: int, hkv: int, dim: int) -> int:
    """Bytes of workspace with which ar_attn_decode spreads its keys over the
    device (zero-initialised once by the caller)."""
    return int(lib().ar_attn_decode_workspace(int(seqs), int(hq), int(hkv), int(dim)))


def _table(table, seqs: int):
    if table.dim() != 2 or table.shape[0] != seqs:
        raise ValueError(f"table must have shape ({seqs}, pages), not {tuple(table.shape)}")
    _typed(table, _I32, "table")
    ptr, ld = _mat(table, (4,), "table")
    return ptr, ld, int(table.shape[1])


def ar_attn_decode(q, cache, table, lens, out, scale=None, window: int = 0, sinks: int = 0, lse=None, workspace=None,
                   stream=None) -> None:
    """Attention of one new token a sequence: q and out [seqs, hq, dim], the
    sequence's keys (its own among them) in the cache's pages `table[seq]`
    (int32), lens[seq] of them.  window 0: no window; scale None: dim ** -0.5.
    attn_decode_workspace(...) zeroed bytes spread the keys over the device."""
    qp = _heads(q, "q")
    seqs, hq, dim = q.shape
    op = _heads(out, "out", (seqs, hq, dim))
    cp = _kv_cache(cache)
    if int(cache[0].shape[3]) != dim:
        raise ValueError(f"the cache's dim is {int(cache[0].shape[3])}, q's {dim}")
    tp, ld, pages = _table(table, seqs)
    np_ = _ints(lens, _I32, "lens", seqs)
    sp, sb = _workspace(workspace)
    _here([q, table, lens, out, lse, workspace, *cache])
    _call("ar_attn_decode", qp, cp, tp, ld, pages, np_, seqs, hq, *_mask(scale, dim, window, sinks), op,
          *_lse(lse, (seqs, hq)), sp, sb, _stream(stream))


def ar_attn(q, k, v, cu_q, cu_k, out, scale=None, window: int = 0, sinks: int = 0, lse=None, stream=None) -> None:
    """Attention of ragged sequences: q and out [rows, hq, dim], k and v
    [rows, hkv, dim]; rows cu_q[b] ... cu_q[b + 1] - 1 (int32) are sequence
    b's.  A query sees the keys up to its own position, within `window` (0:
    all) or among the first `sinks`.  lse [rows, hq] binary32, any strides."""
    qp, kp = _heads(q, "q"), _heads(k, "k")
    (rows, hq, dim), (rows_k, hkv) = q.shape, k.shape[:2]
    vp, op = _heads(v, "v", (rows_k, hkv, dim)), _heads(out, "out", (rows, hq, dim))
    if k.shape[2] != dim:
        raise ValueError(f"k must have heads of {dim}, not {k.shape[2]}")
    seqs = int(cu_q.shape[0]) - 1 if cu_q.dim() == 1 else -1
    if seqs < 0:
        raise ValueError("cu_q must have shape (seqs + 1,)")
    qc, kc = _ints(cu_q, _I32, "cu_q", seqs + 1), _ints(cu_k, _I32, "cu_k", seqs + 1)
    _here([q, k, v, cu_q, cu_k, out, lse])
    _call("ar_attn", qp, kp, vp, qc, kc, seqs, rows, rows_k, hq, hkv, dim, *_mask(scale, dim, window, sinks), op,
          *_lse(lse, (rows, hq)), _stream(stream))


def ar_attn_paged(q, cache, table, lens, cu_q, out, scale=None, window: int = 0, sinks: int = 0, lse=None,
                  stream=None) -> None:
    """ar_attn with the keys in a cache's pages (as in ar_attn_decode): the
    queries are the last of each sequence's lens[b] positions."""
    qp = _heads(q, "q")
    rows, hq, dim = q.shape
    op = _heads(out, "out", (rows, hq, dim))
    cp = _kv_cache(cache)
    if int(cache[0].shape[3]) != dim:
        raise ValueError(f"the cache's dim is {int(cache[0].shape[3])}, q's {dim}")
    seqs = int(cu_q.shape[0]) - 1 if cu_q.dim() == 1 else -1
    if seqs < 0:
        raise ValueError("cu_q must have shape (seqs + 1,)")
    tp, ld, pages = _table(table, seqs)
    np_, qc = _ints(lens, _I32, "lens", seqs), _ints(cu_q, _I32, "cu_q", seqs + 1)
    _here([q, table, lens, cu_q, out, lse, *cache])
    _call("ar_attn_paged", qp, cp, tp, ld, pages, np_, qc, seqs, rows, hq, *_mask(scale, dim, window, sinks), op,
          *_lse(lse, (rows, hq)), _stream(stream))


def attn_bwd_workspace(rows_q: int, rows_k: int, seqs: int, hq: int, hkv: int, dim: int, window: int = 0,
                       sinks: int = 0) -> int:
    """Bytes of workspace that ar_attn_bwd needs."""
    return int(lib().ar_attn_bwd_workspace(int(rows_q), int(rows_k), int(seqs), int(hq), int(hkv), int(dim), int(window),
                                           int(sinks)))


def ar_attn_bwd(q, k, v, out, lse, d_out, cu_q, cu_k, dq=None, dk=None, dv=None, workspace=None, scale=None,
                window: int = 0, sinks: int = 0, stream=None) -> None:
    """Gradient of ar_attn: dq, and / or dk and dv (summed over the query heads
    of a key head), from out and lse of ar_attn and the gradient d_out.  Needs
    attn_bwd_workspace(...) bytes."""
    qp, kp = _heads(q, "q"), _heads(k, "k")
    (rows, hq, dim), (rows_k, hkv) = q.shape, k.shape[:2]
    if k.shape[2] != dim:
        raise ValueError(f"k must have heads of {dim}, not {k.shape[2]}")
    shape_q, shape_k = (rows, hq, dim), (rows_k, hkv, dim)
    vp = _heads(v, "v", shape_k)
    op, gp = _heads(out, "out", shape_q), _heads(d_out, "d_out", shape_q)
    if lse is None:
        raise ValueError("lse is needed")
    dqp = None if dq is None else _heads(dq, "dq", shape_q)
    dkp = None if dk is None else _heads(dk, "dk", shape_k)
    dvp = None if dv is None else _heads(dv, "dv", shape_k)
    seqs = int(cu_q.shape[0]) - 1 if cu_q.dim() == 1 else -1
    if seqs < 0:
        raise ValueError("cu_q must have shape (seqs + 1,)")
    qc, kc = _ints(cu_q, _I32, "cu_q", seqs + 1), _ints(cu_k, _I32, "cu_k", seqs + 1)
    sp, sb = _workspace(workspace)
    _here([q, k, v, out, lse, d_out, cu_q, cu_k, dq, dk, dv, workspace])
    _call("ar_attn_bwd", qp, kp, vp, op, *_lse(lse, (rows, hq)), gp, qc, kc, seqs, rows, rows_k, hq, hkv, dim,
          *_mask(scale, dim, window, sinks), dqp, dkp, dvp, sp, sb, _stream(stream))


def ar_err_init(d_err, stream=None) -> None:
    (ep,) = _bufs([d_err], 8, "d_err", 2)
    _call("ar_err_init", ep, _stream(stream))


def ar_set_launch_shape(kind: int, block: int, vec: int, nt_loads: int, stores: int,
                        wg_per_cu: int) -> None:
    """Set the launch shape of one kernel kind (tuning; process-wide).  `stores`
    is the output store policy: 0 plain, 1 non-temporal, 2 SC1 write-through,
    3 SC1 write-through + non-temporal."""
    _check(lib().ar_set_launch_shape(int(kind), int(block), int(vec), int(nt_loads),
                                     int(stores), int(wg_per_cu)), "ar_set_launch_shape")


def ar_get_launch_shape(kind: int) -> tuple:
    """(block, vec, nt_loads, stores, wg_per_cu) of one kernel kind."""
    v = [ctypes.c_int() for _ in range(5)]
    _check(lib().ar_get_launch_shape(int(kind), *[ctypes.byref(x) for x in v]), "ar_get_launch_shape")
    return tuple(x.value for x in v)


_PREPARABLE = frozenset([ar_reduce_oneshot, ar_reduce_2stage, ar_reduce_2stage_static, ar_pack_fused,
                         ar_unpack_fused, ar_unpack_fused_wait, ar_rd_schedule, ar_reduce_ubatch,
                         ar_reduce_ubatch_flags, ar_quantize_fp8, ar_reduce_fp8, ar_err_init])
_PREPARABLE_BLOCK = frozenset([ar_reduce_norm, ar_norm_bwd, ar_quantize_block, ar_gemm_fp8])
_PREPARABLE_ATTN = frozenset([ar_rope_kv, ar_attn_decode, ar_attn, ar_attn_paged, ar_attn_bwd])
