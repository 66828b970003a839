"""ctypes binding of ``include/ub.h`` -- argument marshalling only.

Every function here has the name of the C entry point it calls and does nothing but
convert arguments (ints, tuples, torch tensors -> pointers and sizes) and turn a non-OK
status into :class:`UBError`.  All work runs in the HIP library ``lib/libub.so``; there is
no fallback: importing this module fails if the library has not been built.

Pointers may be given as ints or as objects with ``data_ptr()`` (torch tensors); streams
as ints, ``None`` (the null stream) or objects with a ``cuda_stream`` attribute.
"""

import ctypes
import os

import torch  # noqa: F401  -- load torch's HIP runtime first; the library binds to it

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libub.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is not built; run `python -m chunked_tp_overlap_amd.build` "
        "(the HIP library is required: there is no CPU fallback)")
_lib = ctypes.CDLL(_LIB_PATH)
LIB_PATH = _LIB_PATH

# ---- enums ------------------------------------------------------------------------------
STATUS = {
    0: "UB_OK", 1: "UB_ERR_INVALID_ARG", 2: "UB_ERR_NDIM", 3: "UB_ERR_ZERO_DIM",
    4: "UB_ERR_CAPACITY", 5: "UB_ERR_HIDDEN_MISMATCH", 6: "UB_ERR_TP_DIVISIBILITY",
    7: "UB_ERR_DTYPE", 8: "UB_ERR_UNSUPPORTED", 9: "UB_ERR_BUFFER_TOO_SMALL",
    10: "UB_ERR_NOT_INITIALIZED", 11: "UB_ERR_HIP",
}
UB_OK = 0
UB_DTYPE_BF16, UB_DTYPE_FP16, UB_DTYPE_FP8_E4M3, UB_DTYPE_FP8_E5M2 = 0, 1, 2, 3
UB_RING_EXCHANGE, UB_PIPELINE, UB_BULK = 0, 1, 2
UB_OP_AG, UB_OP_RS = 0, 1
UB_MAX_STREAMS = 8
METHODS = {"ring_exchange": UB_RING_EXCHANGE, "pipeline": UB_PIPELINE, "bulk": UB_BULK}
UB_REDUCE_ASCENDING, UB_REDUCE_RING = 0, 1
REDUCE_ORDERS = {"ascending": UB_REDUCE_ASCENDING, "ring": UB_REDUCE_RING}
UB_ATTN_PROMPT, UB_ATTN_PROMPT_BWD, UB_ATTN_DECODE = 0, 1, 2
UB_ATTN_MAX_HEAD_DIM = 128

# Every symbol include/ub.h declares.
EXPORTS = (
    "ub_overlap_cfg_default", "ub_required_bytes", "ub_init", "ub_set_active_shape",
    "ub_get_active_shape", "ub_get_capacity_shape", "ub_get_plan", "ub_copy_in",
    "ub_gemm_ag_chunked", "ub_gemm_ag_arrival", "ub_arrival_timeouts", "ub_deliver_chunks",
    "ub_quantize_in",
    "ub_gemm_ag_chunked_fp8", "ub_gemm_rs_chunked", "ub_gemm_rs_chunked_noalloc",
    "ub_gemm_rs_chunked_fp8",
    "ub_quantize_e4m3", "ub_reduce_partials",
    "ub_set_kernel_timing", "ub_get_kernel_timing", "ub_prepare_streams", "ub_debug_set",
    "ub_debug_last_plan", "ub_register_scratch", "ub_destroy", "ub_status_string", "ub_last_error",
    "ub_attn_required_bytes", "ub_kv_append", "ub_attn_prompt", "ub_attn_prompt_bwd", "ub_attn_decode",
)


class UBError(RuntimeError):
    def __init__(self, status, message=""):
        self.status = status
        self.name = STATUS.get(status, f"UB_ERR_{status}")
        super().__init__(f"{self.name}: {message}" if message else self.name)


# ---- structs ----------------------------------------------------------------------------
class ub_overlap_cfg_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "method", "num_splits", "num_max_streams", "aggregate", "atomic_gemm", "rank",
        "use_ce", "num_sm", "set_sm_margin", "reduce_order", "fuse_reduce")]


class ub_plan_unit_t(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_int32), ("unit", ctypes.c_int32), ("row0", ctypes.c_int64),
                ("row1", ctypes.c_int64), ("stream", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ub_tile_plan_t(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("cut_row", ctypes.c_int64),
                ("tail_tile_m", ctypes.c_int32), ("tail_tile_n", ctypes.c_int32),
                ("seg_row", ctypes.c_int64), ("nseg", ctypes.c_int32), ("split", ctypes.c_int32),
                ("seg_tile_m", ctypes.c_int32), ("seg_tile_n", ctypes.c_int32),
                ("dispatches", ctypes.c_int32), ("rs_pieces", ctypes.c_int32)]


class ub_attn_cfg_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_heads", "n_kv_heads", "head_dim", "rotary_dim",
                                              "rope_interleaved")] + [("softmax_scale", ctypes.c_float)]


class ub_heads_t(ctypes.Structure):
    tensor = held = None  # what heads() describes; the (heads, dim) it was last checked against
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("rows", ctypes.c_int64)]


class ub_kv_cache_t(ctypes.Structure):
    tensors, held = (), None
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


UB_SCRATCH_COUNTER_BYTES = 256 * 1024
UB_SCRATCH_MIN_BYTES = UB_SCRATCH_COUNTER_BYTES + 64 * 1024


class ub_kernel_stats_t(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int64), ("total_ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


_H = ctypes.c_void_p
_P = ctypes.c_void_p
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_CFGP = ctypes.POINTER(ub_overlap_cfg_t)

_ATTNP, _HEADSP, _KVP = (ctypes.POINTER(t) for t in (ub_attn_cfg_t, ub_heads_t, ub_kv_cache_t))

_sig = {
    "ub_overlap_cfg_default": (None, [_CFGP]),
    "ub_required_bytes": (_I32, [_I64, _I64, _I32, _I32, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "ub_init": (_I32, [ctypes.POINTER(_H), _I64, _I64, _I32, _I32, _P, _SZ, _P, _SZ]),
    "ub_set_active_shape": (_I32, [_H, ctypes.POINTER(_I64), _I32]),
    "ub_get_active_shape": (_I32, [_H, ctypes.POINTER(_I64)]),
    "ub_get_capacity_shape": (_I32, [_H, ctypes.POINTER(_I64)]),
    "ub_get_plan": (_I32, [_H, _CFGP, _I32, ctypes.POINTER(ub_plan_unit_t), _I32,
                           ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "ub_copy_in": (_I32, [_H, _P, _I64, _I64, _P]),
    "ub_gemm_ag_chunked": (_I32, [_H, _P, _I64, _I64, _P, _I64, _CFGP, _P]),
    "ub_gemm_ag_arrival": (_I32, [_H, _P, _I32, _P, _I64, _I64, _P, _I64, _CFGP, _P]),
    "ub_deliver_chunks": (_I32, [_H, _P, _I32, _CFGP, _P]),
    "ub_arrival_timeouts": (_I32, [_H, ctypes.POINTER(ctypes.c_uint32)]),
    "ub_quantize_in": (_I32, [_H, _P, _I64, _I64, ctypes.c_float, _P]),
    "ub_gemm_ag_chunked_fp8": (_I32, [_H, _P, _I64, _I64, ctypes.c_float, ctypes.c_float, _P,
                                      _I64, _CFGP, _P]),
    "ub_gemm_rs_chunked": (_I32, [_H, _P, _I64, _I64, _P, _I64, _P, _I64, _CFGP, _P]),
    "ub_gemm_rs_chunked_noalloc": (_I32, [_H, _P, _I64, _I64, _P, _I64, _P, _I64, _CFGP, _P]),
    "ub_gemm_rs_chunked_fp8": (_I32, [_H, _P, _I64, _I64, _P, _I64, ctypes.c_float, ctypes.c_float,
                                      _P, _I64, _CFGP, _P]),
    "ub_quantize_e4m3": (_I32, [_P, _I64, _P, _I64, _I64, _I64, ctypes.c_float, _P]),
    "ub_reduce_partials": (_I32, [_H, _P, _I64, _I32, _P]),
    "ub_set_kernel_timing": (_I32, [_H, _I32]),
    "ub_get_kernel_timing": (_I32, [_H, ctypes.POINTER(ub_kernel_stats_t),
                                    ctypes.POINTER(ub_kernel_stats_t)]),
    "ub_prepare_streams": (_I32, [_H, _I32, _I32]),
    "ub_debug_set": (_I32, [_H, ctypes.c_char_p, _I64]),
    "ub_debug_last_plan": (_I32, [_H, ctypes.POINTER(ub_tile_plan_t)]),
    "ub_register_scratch": (_I32, [_H, _P, _SZ]),
    "ub_attn_required_bytes": (_I32, [_I32, _ATTNP, _I64, _I32, ctypes.POINTER(_SZ)]),
    "ub_kv_append": (_I32, [_H, _HEADSP, _HEADSP, _HEADSP, _HEADSP, _HEADSP, _P, _P, _P, _I32, _KVP, _P,
                            _I64, _I32, _ATTNP, _P]),
    "ub_attn_prompt": (_I32, [_H, _HEADSP, _HEADSP, _HEADSP, _HEADSP, _P, _P, _I32, _ATTNP, _P, _SZ, _P]),
    "ub_attn_prompt_bwd": (_I32, [_H] + [_HEADSP] * 5 + [_P] + [_HEADSP] * 3 + [_P, _I32, _ATTNP, _P, _SZ, _P]),
    "ub_attn_decode": (_I32, [_H, _HEADSP, _KVP, _P, _I64, _I32, _P, _I32, _HEADSP, _P, _ATTNP, _P, _SZ, _P]),
    "ub_destroy": (_I32, [_H]),
    "ub_status_string": (ctypes.c_char_p, [_I32]),
    "ub_last_error": (ctypes.c_char_p, [_H]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


# ---- marshalling helpers ------------------------------------------------------------------
def _ptr(x):
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _stream(s):
    if s is None:
        return None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def _check(st, h=None):
    if st != UB_OK:
        raise UBError(st, ub_last_error(h) if h else "")


def ub_status_string(status):
    return _lib.ub_status_string(int(status)).decode()


def ub_last_error(h):
    return (_lib.ub_last_error(h) or b"").decode()


def ub_overlap_cfg_default():
    cfg = ub_overlap_cfg_t()
    _lib.ub_overlap_cfg_default(ctypes.byref(cfg))
    return cfg


def _reduce_order(x):
    return REDUCE_ORDERS[x] if isinstance(x, str) else int(x)


def make_cfg(method="ring_exchange", num_splits=1, num_max_streams=3, aggregate=False,
             atomic_gemm=False, rank=0, use_ce=True, num_sm=0, set_sm_margin=False,
             reduce_order="ascending", fuse_reduce=False):
    """A ``ub_overlap_cfg_t`` from keyword options ([TE#1344] option names, plus the
    reduce-scatter summation order "ascending" or "ring" and whether the reduce-scatter
    sum runs inside the slice-GEMM launch)."""
    cfg = ub_overlap_cfg_default()
    cfg.method = METHODS[method] if isinstance(method, str) else int(method)
    cfg.num_splits = int(num_splits)
    cfg.num_max_streams = int(num_max_streams)
    cfg.aggregate = int(bool(aggregate))
    cfg.atomic_gemm = int(bool(atomic_gemm))
    cfg.rank = int(rank)
    cfg.use_ce = int(bool(use_ce))
    cfg.num_sm = int(num_sm)
    cfg.set_sm_margin = int(bool(set_sm_margin))
    cfg.reduce_order = _reduce_order(reduce_order)
    cfg.fuse_reduce = int(bool(fuse_reduce))
    return cfg


def ub_required_bytes(capacity, hidden, tp_size, dtype=UB_DTYPE_BF16):
    a, b = _SZ(), _SZ()
    _check(_lib.ub_required_bytes(capacity, hidden, tp_size, dtype, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def _fits(buf, nbytes, what):
    """A tensor passed with a byte count must hold that many bytes (the library trusts the
    count and addresses up to it)."""
    if hasattr(buf, "numel") and hasattr(buf, "element_size"):
        have = buf.numel() * buf.element_size()
        if int(nbytes) > have:
            raise ValueError(f"{what}: {int(nbytes)} bytes declared, the tensor holds {have}")


def ub_init(capacity, hidden, tp_size, dtype, ub_buf, ub_bytes, rs_ws=None, rs_ws_bytes=0):
    _fits(ub_buf, ub_bytes, "ub_buf")
    if rs_ws is not None:
        _fits(rs_ws, rs_ws_bytes, "rs_ws")
    h = _H()
    _check(_lib.ub_init(ctypes.byref(h), capacity, hidden, tp_size, dtype, _ptr(ub_buf),
                        int(ub_bytes), _ptr(rs_ws), int(rs_ws_bytes)))
    return h


def ub_set_active_shape(h, shape, check=True):
    """Returns the status code; raises UBError on failure when ``check``."""
    arr = (_I64 * max(len(shape), 1))(*[int(d) for d in shape])
    st = _lib.ub_set_active_shape(h, arr, len(shape))
    if check:
        _check(st, h)
    return st


def ub_get_active_shape(h):
    out = (_I64 * 2)()
    _check(_lib.ub_get_active_shape(h, out), h)
    return (out[0], out[1])


def ub_get_capacity_shape(h):
    out = (_I64 * 2)()
    _check(_lib.ub_get_capacity_shape(h, out), h)
    return (out[0], out[1])


def ub_get_plan(h, cfg, op=UB_OP_AG, max_units=4096):
    """Returns (list of (pos, unit, row0, row1, stream), n_streams)."""
    buf = (ub_plan_unit_t * max_units)()
    n, s = _I32(), _I32()
    _check(_lib.ub_get_plan(h, ctypes.byref(cfg), op, buf, max_units, ctypes.byref(n), ctypes.byref(s)), h)
    units = [(u.pos, u.unit, u.row0, u.row1, u.stream) for u in buf[: min(n.value, max_units)]]
    return units, s.value


def ub_copy_in(h, src, rows, row_offset, stream=None):
    _check(_lib.ub_copy_in(h, _ptr(src), rows, row_offset, _stream(stream)), h)


def ub_gemm_ag_chunked(h, w, n_cols, ldw, c, ldc, cfg, stream=None):
    _check(_lib.ub_gemm_ag_chunked(h, _ptr(w), n_cols, ldw, _ptr(c), ldc, ctypes.byref(cfg),
                                   _stream(stream)), h)


def _on_host(src):
    return int(hasattr(src, "is_cuda") and not src.is_cuda)


def ub_gemm_ag_arrival(h, src, w, n_cols, ldw, c, ldc, cfg, stream=None):
    """src: a device tensor, or a pinned host tensor (then delivered over PCIe)."""
    _check(_lib.ub_gemm_ag_arrival(h, _ptr(src), _on_host(src), _ptr(w), n_cols, ldw, _ptr(c),
                                   ldc, ctypes.byref(cfg), _stream(stream)), h)


def ub_deliver_chunks(h, src, cfg, stream=None):
    _check(_lib.ub_deliver_chunks(h, _ptr(src), _on_host(src), ctypes.byref(cfg),
                                  _stream(stream)), h)


def ub_arrival_timeouts(h):
    """Tile waits of the arrival-gated device-side chunk loop that hit the time bound."""
    n = ctypes.c_uint32(0)
    _check(_lib.ub_arrival_timeouts(h, ctypes.byref(n)), h)
    return n.value


def ub_quantize_in(h, src, rows, row_offset, scale, stream=None):
    _check(_lib.ub_quantize_in(h, _ptr(src), rows, row_offset, float(scale), _stream(stream)), h)


def ub_gemm_ag_chunked_fp8(h, w, n_cols, ldw, scale_inv_a, scale_inv_w, c, ldc, cfg, stream=None):
    _check(_lib.ub_gemm_ag_chunked_fp8(h, _ptr(w), n_cols, ldw, float(scale_inv_a),
                                       float(scale_inv_w), _ptr(c), ldc, ctypes.byref(cfg),
                                       _stream(stream)), h)


def ub_gemm_rs_chunked(h, a, k, lda, w, ldw, out, ldo, cfg, stream=None):
    _check(_lib.ub_gemm_rs_chunked(h, _ptr(a), k, lda, _ptr(w), ldw, _ptr(out), ldo,
                                   ctypes.byref(cfg), _stream(stream)), h)


def ub_gemm_rs_chunked_noalloc(h, a, k, lda, w, ldw, out, ldo, cfg, stream=None):
    _check(_lib.ub_gemm_rs_chunked_noalloc(h, _ptr(a), k, lda, _ptr(w), ldw, _ptr(out), ldo,
                                   ctypes.byref(cfg), _stream(stream)), h)


def ub_gemm_rs_chunked_fp8(h, a, k, lda, w, ldw, scale_inv_a, scale_inv_w, out, ldo, cfg,
                           stream=None):
    """a: [T, k] E4M3 codes (row stride lda bytes); w: [hidden, k] E4M3 codes (row stride
    ldw bytes); out: [T, hidden] bf16 (row stride ldo elements)."""
    _check(_lib.ub_gemm_rs_chunked_fp8(h, _ptr(a), k, lda, _ptr(w), ldw, float(scale_inv_a),
                                       float(scale_inv_w), _ptr(out), ldo, ctypes.byref(cfg),
                                       _stream(stream)), h)


def ub_quantize_e4m3(src, lds, dst, ldd, rows, cols, scale, stream=None):
    """dst [rows, cols] E4M3 (row stride ldd bytes) = quantized src (bf16, row stride lds)."""
    _check(_lib.ub_quantize_e4m3(_ptr(src), lds, _ptr(dst), ldd, rows, cols, float(scale),
                                 _stream(stream)))


def ub_reduce_partials(h, out, ldo, reduce_order="ascending", stream=None):
    _check(_lib.ub_reduce_partials(h, _ptr(out), ldo, _reduce_order(reduce_order),
                                   _stream(stream)), h)


def ub_set_kernel_timing(h, enable):
    """enable: False/0 off, True/1 an event pair per launch, 2 chained (one event per launch)."""
    _check(_lib.ub_set_kernel_timing(h, int(enable)), h)


def ub_get_kernel_timing(h):
    """Returns (gemm, reduce) dicts: launches, total_ms, flops, bytes."""
    g, r = ub_kernel_stats_t(), ub_kernel_stats_t()
    _check(_lib.ub_get_kernel_timing(h, ctypes.byref(g), ctypes.byref(r)), h)
    conv = lambda s: {"launches": s.launches, "total_ms": s.total_ms, "flops": s.flops, "bytes": s.bytes}
    return conv(g), conv(r)


def ub_prepare_streams(h, num_max_streams=3, copy_stream=False):
    _check(_lib.ub_prepare_streams(h, int(num_max_streams), int(bool(copy_stream))), h)


def ub_debug_set(h, key, value):
    _check(_lib.ub_debug_set(h, key.encode(), int(value)), h)


def ub_debug_last_plan(h, seg=False):
    """(tile_m, tile_n, cut_row, tail_tile_m, tail_tile_n) of the last GEMM launch group, and
    with seg=True also (seg_row, nseg, split, seg_tile_m, seg_tile_n)."""
    p = ub_tile_plan_t()
    _check(_lib.ub_debug_last_plan(h, ctypes.byref(p)), h)
    base = (p.tile_m, p.tile_n, p.cut_row, p.tail_tile_m, p.tail_tile_n)
    return base + (p.seg_row, p.nseg, p.split, p.seg_tile_m, p.seg_tile_n) if seg else base


def ub_debug_plan(h):
    """Every field of the last call's plan record as a dict."""
    p = ub_tile_plan_t()
    _check(_lib.ub_debug_last_plan(h, ctypes.byref(p)), h)
    return {name: getattr(p, name) for name, _ in ub_tile_plan_t._fields_}


def ub_register_scratch(h, buf, nbytes):
    if buf is not None:
        _fits(buf, nbytes, "scratch")
    _check(_lib.ub_register_scratch(h, _ptr(buf), int(nbytes)), h)


# ---- attention ----------------------------------------------------------------------------
def make_attn_cfg(n_heads, n_kv_heads, head_dim, rotary_dim=None, rope_interleaved=False,
                  softmax_scale=None):
    """A ``ub_attn_cfg_t``; rotary_dim defaults to head_dim rounded down to a multiple of 16,
    softmax_scale to head_dim ** -0.5."""
    cfg = ub_attn_cfg_t()
    cfg.n_heads, cfg.n_kv_heads, cfg.head_dim = int(n_heads), int(n_kv_heads), int(head_dim)
    cfg.rotary_dim = int(head_dim) // 16 * 16 if rotary_dim is None else int(rotary_dim)
    cfg.rope_interleaved = int(bool(rope_interleaved))
    cfg.softmax_scale = max(int(head_dim), 1) ** -0.5 if softmax_scale is None else float(softmax_scale)
    return cfg


def heads(x, col=0):
    """A ``ub_heads_t`` over a bf16 device tensor: the heads that start at column ``col`` of a 2-D
    [rows, columns] matrix, head_dim columns each, or a 3-D [rows, heads, head_dim] view with
    any row and head strides of head_dim and more.  It keeps the tensor alive."""
    if x.dim() not in (2, 3):
        raise ValueError(f"heads: a 2-D or 3-D tensor, not {x.dim()}-D")
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"heads: a bf16 matrix, not {x.dtype}")
    if x.numel() and x.stride(-1) != 1:
        raise ValueError("heads: the last dimension must be contiguous")
    if x.dim() == 3 and col:
        raise ValueError("heads: col is for 2-D matrices")
    if col < 0:
        raise ValueError(f"heads: col {col} lies before the matrix")
    if x.dim() == 3 and x.shape[1] > 1 and x.stride(1) == 0:
        raise ValueError("heads: one head expanded to several; a head stride of 0 stands for head_dim")
    d = ub_heads_t()
    d.ptr = x.data_ptr() + 2 * int(col)
    d.rows = x.shape[0]
    d.row_stride = x.stride(0)
    d.head_stride = x.stride(1) if x.dim() == 3 else 0
    d.tensor, d.col = x, int(col)
    return d


def make_kv_cache(k, v, k_scale=1.0, v_scale=1.0):
    """A ``ub_kv_cache_t`` over k and v, [n_pages, kv_heads, page_size, head_dim] views of the
    same strides (any order of heads and tokens), bf16, or float8_e4m3fn with the scales."""
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
        raise ValueError("make_kv_cache: k and v must be 4-D, of one shape, dtype and strides")
    if k.stride(3) != 1:
        raise ValueError("make_kv_cache: head_dim must be contiguous")
    dtypes = {torch.bfloat16: UB_DTYPE_BF16, torch.float8_e4m3fn: UB_DTYPE_FP8_E4M3,
              torch.float16: UB_DTYPE_FP16, torch.float8_e5m2: UB_DTYPE_FP8_E5M2}
    if k.dtype not in dtypes:
        raise ValueError(f"make_kv_cache: {k.dtype}")
    c = ub_kv_cache_t()
    c.k, c.v = k.data_ptr(), v.data_ptr()
    c.page_stride, c.head_stride, c.token_stride = k.stride(0), k.stride(1), k.stride(2)
    c.n_pages, c.page_size = k.shape[0], k.shape[2]
    c.dtype = dtypes[k.dtype]
    c.k_scale, c.v_scale = float(k_scale), float(v_scale)
    c.tensors = (k, v)
    return c


# A call's own cost is a few microseconds, as much as a small batch's kernel: descriptors are
# checked against a head layout once, and tensors with as few attribute reads as it takes.
def _host(x, what):
    """Refuses a tensor of pageable host memory, which no kernel can address."""
    if not x.is_pinned():
        raise ValueError(f"{what}: a device tensor, not one in host memory")


def _hold_heads(x, layout, what):
    """Checks that x's columns hold the (heads, dim) of layout."""
    n, D = layout
    t = x.tensor
    if t is not None:
        if t.dim() == 3 and (t.shape[1] < n or t.shape[2] < D):
            raise ValueError(f"{what}: {tuple(t.shape)} does not hold {n} heads of {D}")
        if t.dim() == 2 and x.col + n * D > t.shape[1]:
            raise ValueError(f"{what}: columns {x.col} to {x.col + n * D} of {t.shape[1]}")
        if not t.is_cuda:
            _host(t, what)
        x.held = layout


def _hold_cache(cache, layout):
    n, D = layout
    for t in cache.tensors:
        if t.shape[1] < n or t.shape[3] < D:
            raise ValueError(f"cache: {tuple(t.shape)} does not hold {n} heads of {D}")
        if not t.is_cuda:
            _host(t, "cache")
    if cache.tensors:
        cache.held = layout


def _int32(x, n, what):
    """A pointer to at least n contiguous int32 values."""
    if type(x) is torch.Tensor or isinstance(x, torch.Tensor):
        if x.dtype is not torch.int32 or x.numel() < n or not x.is_contiguous():
            raise ValueError(f"{what}: at least {n} contiguous int32 values")
        if not x.is_cuda:
            _host(x, what)
        return x.data_ptr()
    return _ptr(x)


def _table(pages, n):
    """(pointer, row stride, pages per sequence) of a [sequences, pages] int32 tensor."""
    if pages is None:
        return None, 0, 0
    shape = pages.shape
    if len(shape) == 2 and pages.dtype is torch.int32:
        rows, per = shape
        ld, one = pages.stride()
        # the stride of a single row means nothing; rows that overlap (an expanded one among them)
        # are not what the calls read
        if rows >= n and (one == 1 or rows * per == 0) and (ld >= per or n <= 1):
            if not pages.is_cuda:
                _host(pages, "pages")
            return pages.data_ptr(), ld if ld > per else per, per
    raise ValueError(f"pages: an int32 [at least {n}, pages] tensor with contiguous rows that do not overlap")


def _lse_arg(lse, h, cfg, out):
    """A call needs n_heads T values.  It refuses an `out` of fewer than T rows, so as many per
    row of `out` are enough; asking the handle for T costs a call of its own."""
    if type(lse) is torch.Tensor or isinstance(lse, torch.Tensor):
        n, H = lse.numel(), cfg.n_heads
        if lse.dtype is not torch.float32 or not lse.is_contiguous() or \
                ((out is None or n < H * out.rows) and n < H * ub_get_active_shape(h)[0]):
            raise ValueError(f"lse: a contiguous float32 [{H}, {ub_get_active_shape(h)[0]}] tensor")
        if not lse.is_cuda:
            _host(lse, "lse")
        return lse.data_ptr()
    return _ptr(lse)


def _ws_arg(ws):
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("workspace: a contiguous tensor")
    if not ws.is_cuda:
        _host(ws, "workspace")
    return ws.data_ptr(), ws.nbytes


def ub_attn_required_bytes(op, cfg, rows, n_seqs):
    n = _SZ()
    _check(_lib.ub_attn_required_bytes(int(op), ctypes.byref(cfg), rows, n_seqs, ctypes.byref(n)))
    return n.value


def ub_kv_append(h, q, k, v, q_out, k_out, inv_freq, cu_seqlens, past_lens, n_seqs, cache, pages, cfg,
                 stream=None):
    """q, k, v, q_out, k_out: ``heads(...)`` or None; cache: ``make_kv_cache(...)`` or None; pages:
    a [sequences, pages] int32 tensor; inv_freq: rotary_dim / 2 floats."""
    D = cfg.head_dim
    H, G = (cfg.n_heads, D), (cfg.n_kv_heads, D)
    if q is not None and q.held != H:
        _hold_heads(q, H, "q")
    if k is not None and k.held != G:
        _hold_heads(k, G, "k")
    if v is not None and v.held != G:
        _hold_heads(v, G, "v")
    if q_out is not None and q_out.held != H:
        _hold_heads(q_out, H, "q_out")
    if k_out is not None and k_out.held != G:
        _hold_heads(k_out, G, "k_out")
    if cache is not None and cache.held != G:
        _hold_cache(cache, G)
    if type(inv_freq) is torch.Tensor or isinstance(inv_freq, torch.Tensor):
        if inv_freq.dtype is not torch.float32 or not inv_freq.is_contiguous() \
                or inv_freq.numel() < cfg.rotary_dim // 2:
            raise ValueError(f"inv_freq: at least {cfg.rotary_dim // 2} contiguous float32 values")
        if not inv_freq.is_cuda:
            _host(inv_freq, "inv_freq")
        inv_freq = inv_freq.data_ptr()
    else:
        inv_freq = _ptr(inv_freq)
    table, ld, per_seq = _table(pages, n_seqs)
    st = _lib.ub_kv_append(h, q, k, v, q_out, k_out, inv_freq, _int32(cu_seqlens, n_seqs + 1, "cu_seqlens"),
                           _int32(past_lens, n_seqs, "past_lens"), n_seqs, cache, table, ld, per_seq, cfg,
                           _stream(stream))
    if st:
        _check(st, h)


def ub_attn_prompt(h, q, k, v, out, lse, cu_seqlens, n_seqs, cfg, workspace=None, stream=None):
    D = cfg.head_dim
    H, G = (cfg.n_heads, D), (cfg.n_kv_heads, D)
    for x, layout, what in ((q, H, "q"), (k, G, "k"), (v, G, "v"), (out, H, "out")):
        if x is not None and x.held != layout:
            _hold_heads(x, layout, what)
    ws, ws_bytes = _ws_arg(workspace)
    st = _lib.ub_attn_prompt(h, q, k, v, out, _lse_arg(lse, h, cfg, out), _int32(cu_seqlens, n_seqs + 1, "cu_seqlens"),
                             n_seqs, cfg, ws, ws_bytes, _stream(stream))
    if st:
        _check(st, h)


def ub_attn_prompt_bwd(h, dout, q, k, v, out, lse, dq, dk, dv, cu_seqlens, n_seqs, cfg, workspace,
                       stream=None):
    D = cfg.head_dim
    H, G = (cfg.n_heads, D), (cfg.n_kv_heads, D)
    for x, layout, what in ((dout, H, "dout"), (q, H, "q"), (k, G, "k"), (v, G, "v"), (out, H, "out"), (dq, H, "dq"),
                            (dk, G, "dk"), (dv, G, "dv")):
        if x is not None and x.held != layout:
            _hold_heads(x, layout, what)
    ws, ws_bytes = _ws_arg(workspace)
    st = _lib.ub_attn_prompt_bwd(h, dout, q, k, v, out, _lse_arg(lse, h, cfg, out), dq, dk, dv,
                                 _int32(cu_seqlens, n_seqs + 1, "cu_seqlens"), n_seqs, cfg, ws, ws_bytes,
                                 _stream(stream))
    if st:
        _check(st, h)


def ub_attn_decode(h, q, cache, pages, kv_lens, n_seqs, out, lse, cfg, workspace, stream=None):
    D = cfg.head_dim
    H, G = (cfg.n_heads, D), (cfg.n_kv_heads, D)
    if q is not None and q.held != H:
        _hold_heads(q, H, "q")
    if out is not None and out.held != H:
        _hold_heads(out, H, "out")
    if cache is not None and cache.held != G:
        _hold_cache(cache, G)
    table, ld, per_seq = _table(pages, n_seqs)
    ws, ws_bytes = _ws_arg(workspace)
    st = _lib.ub_attn_decode(h, q, cache, table, ld, per_seq, _int32(kv_lens, n_seqs, "kv_lens"), n_seqs, out,
                             _lse_arg(lse, h, cfg, out), cfg, ws, ws_bytes, _stream(stream))
    if st:
        _check(st, h)


def ub_destroy(h):
    _check(_lib.ub_destroy(h))


def raw_call(name, *args):
    """Call a C entry point with already-marshalled arguments and return its raw status
    (for tests of the error paths)."""
    return getattr(_lib, name)(*args)
