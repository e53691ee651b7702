"""Python binding of the MI355X mixed-precision partial-sum reduce (``include/ar.h``).

Argument marshalling only: every step of the reduce runs in the HIP library
``libmpp_ar.so`` built from ``csrc/`` for gfx950.  The binding loads that
library and nothing else; if it is missing, importing succeeds but the first
call raises ``RuntimeError`` -- there is no fallback path.

The functions carry the C names:

    ctx = ar_init(device=0, config=None)
    ar_reduce(ctx, dsts, srcs, n, dst_type, wire_type, mode, stream=None)
    ar_reduce_add(ctx, dsts, srcs, n, dst_type, wire_type, mode, residual, residual_len, stream=None)
    ar_reduce_rows(ctx, dsts, srcs, rows, cols, src_stride, dst_stride, dst_type, wire_type, mode,
                   residual=None, res_stride=0, stream=None)
    ar_qk_norm_rope(ctx, q, k, q_weight, k_weight, table, positions, ...)
    ar_attention(ctx, out, q, k, v, cu_q, k_start, k_len, max_q, max_k, ...)
    ar_fp8_quantize(ctx, codes, scales, x)
    ar_fp8_matmul(ctx, out, a, a_scales, b, b_scales, ...)
    ar_free(ctx)
    ar_status_str(code)
    ar_plan_query(...), ar_plan_query_add(...), ar_plan_query_rows(...)

``dsts`` / ``srcs`` are sequences of torch tensors or raw integer addresses, or
ready-made ``ptr_array(...)`` arrays (passed through unchanged, which keeps
the per-call marshalling cost low for latency-bound callers); ``stream`` is a
``torch.cuda.Stream``, a raw ``hipStream_t`` integer, or None for the null
stream (for the layer operators torch's current stream).

The library sees only pointers, so it cannot tell how large a buffer is.  With
``validate=True`` (the default) the enqueueing calls check, before calling it,
that every tensor argument spans the bytes the call will read or write from its
data pointer (and, for the 1-D calls, that it is contiguous), raising
``ValueError`` otherwise; integer addresses and ``ptr_array`` arrays are the
caller's responsibility, as in C.  ``bind_reduce`` and ``bind_reduce_rows`` check once,
when they bind.

The layer operators (``ar_qk_norm_rope`` to ``ar_fp8_matmul``) take torch tensors
only: types, sizes and strides come from them, and a tensor that does not fit
raises ``ValueError`` before the call.  Without a ``stream`` they are enqueued, as
torch's own operations are, on torch's current stream of the tensors' device.
With one, torch's allocator does not know of the work there: a tensor made on
another stream is kept until that work is done (or told with ``record_stream``).
"""
from __future__ import annotations

import ctypes
import os

AR_F32, AR_F16, AR_BF16 = 0, 1, 2
AR_MODE_AUTO, AR_MODE_SINGLE_SHOT, AR_MODE_CHUNKED, AR_MODE_RS_BCAST, AR_MODE_HOST_STAGED = 0, 1, 2, 3, 4
AR_MODE_MASK = 0xFF
AR_SRC_WIRE = 0x100
AR_SRC_INACTIVE_NULL = 0x200
AR_MAX_RANKS = 16
AR_QK_INTERLEAVED = 0x1
AR_ATTN_CAUSAL = 0x1
AR_F8_BLOCK = 128

AR_OK, AR_ERR_INVALID, AR_ERR_UNSUPPORTED, AR_ERR_NOMEM, AR_ERR_RUNTIME = 0, 1, 2, 3, 4

MODE_NAMES = {
    AR_MODE_AUTO: "auto", AR_MODE_SINGLE_SHOT: "single_shot", AR_MODE_CHUNKED: "chunked",
    AR_MODE_RS_BCAST: "rs_bcast", AR_MODE_HOST_STAGED: "host_staged",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmpp_ar.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "ar.h")


class ArConfig(ctypes.Structure):
    _fields_ = [
        ("single_shot_max_bytes", ctypes.c_size_t),
        ("chunk_bytes", ctypes.c_size_t),
        ("host_chunk_bytes", ctypes.c_size_t),
        ("host_slots", ctypes.c_int),
        ("grid_wgs", ctypes.c_int),
        ("stream_kernel", ctypes.c_int),
        ("store_policy", ctypes.c_int),
        ("host_path", ctypes.c_int),
        ("xcd_run_elems", ctypes.c_size_t),
        ("occupancy_hold", ctypes.c_int),
    ]


class ArPlan(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int),
        ("n_dst", ctypes.c_int),
        ("src_bytes", ctypes.c_int),
        ("wire_bytes", ctypes.c_int),
        ("chunk_elems", ctypes.c_size_t),
        ("n_chunks", ctypes.c_size_t),
        ("slice_start", ctypes.c_size_t * AR_MAX_RANKS),
        ("slice_len", ctypes.c_size_t * AR_MAX_RANKS),
        ("algo_bytes", ctypes.c_size_t),
        ("store_nt", ctypes.c_int),
        ("host_direct", ctypes.c_int),
        ("stream_kernel", ctypes.c_int),
        ("active_mask", ctypes.c_uint),
        ("dst_bytes", ctypes.c_int),
        ("residual_kind", ctypes.c_int),
        ("hold_waves", ctypes.c_int),
    ]


class ArRows(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_size_t),
        ("cols", ctypes.c_size_t),
        ("src_stride", ctypes.c_size_t),
        ("dst_stride", ctypes.c_size_t),
        ("res_stride", ctypes.c_size_t),
    ]


class ArQk(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_size_t),
        ("heads_q", ctypes.c_int), ("heads_kv", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int),
        ("q_token", ctypes.c_size_t), ("q_head", ctypes.c_size_t),
        ("k_token", ctypes.c_size_t), ("k_head", ctypes.c_size_t),
        ("v_token", ctypes.c_size_t), ("v_head", ctypes.c_size_t),
        ("q_out_token", ctypes.c_size_t), ("q_out_head", ctypes.c_size_t),
        ("k_out_token", ctypes.c_size_t), ("k_out_head", ctypes.c_size_t),
        ("v_out_token", ctypes.c_size_t), ("v_out_head", ctypes.c_size_t),
        ("table_rows", ctypes.c_size_t), ("cache_rows", ctypes.c_size_t),
        ("eps", ctypes.c_float), ("flags", ctypes.c_uint),
    ]


class ArAttn(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("heads_q", ctypes.c_int), ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("total_q", ctypes.c_size_t), ("rows_k", ctypes.c_size_t),
        ("max_q", ctypes.c_int), ("max_k", ctypes.c_int),
        ("q_token", ctypes.c_size_t), ("q_head", ctypes.c_size_t),
        ("k_token", ctypes.c_size_t), ("k_head", ctypes.c_size_t),
        ("v_token", ctypes.c_size_t), ("v_head", ctypes.c_size_t),
        ("o_token", ctypes.c_size_t), ("o_head", ctypes.c_size_t),
        ("scale", ctypes.c_float), ("flags", ctypes.c_uint),
    ]


class ArMm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("rows", "cols", "depth", "a_row", "b_row", "out_row")]


class ArError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {ar_status_str(status)} ({status})" if what else ar_status_str(status))


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmpp_ar.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"HIP library {path} is missing: build it with "
            "`python -m mixed_precision_partial_amd.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.ar_init.argtypes = [ctypes.POINTER(vp), ctypes.c_int, ctypes.POINTER(ArConfig)]
    lib.ar_init.restype = ctypes.c_int
    lib.ar_reduce.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_int, sz,
                              ctypes.c_int, ctypes.c_int, ctypes.c_uint, vp]
    lib.ar_reduce.restype = ctypes.c_int
    lib.ar_reduce_staged_static.argtypes = lib.ar_reduce.argtypes
    lib.ar_reduce_staged_static.restype = ctypes.c_int
    lib.ar_free.argtypes = [vp]
    lib.ar_free.restype = ctypes.c_int
    lib.ar_status_str.argtypes = [ctypes.c_int]
    lib.ar_status_str.restype = ctypes.c_char_p
    lib.ar_plan_query.argtypes = [ctypes.POINTER(ArConfig), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                  ctypes.c_int, sz, ctypes.c_int, ctypes.c_int, ctypes.c_uint,
                                  ctypes.c_int, ctypes.POINTER(ArPlan)]
    lib.ar_plan_query.restype = ctypes.c_int
    lib.ar_reduce_add.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_int, sz,
                                  ctypes.c_int, ctypes.c_int, ctypes.c_uint, vp, sz, vp]
    lib.ar_reduce_add.restype = ctypes.c_int
    lib.ar_plan_query_add.argtypes = [ctypes.POINTER(ArConfig), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                      ctypes.c_int, sz, ctypes.c_int, ctypes.c_int, ctypes.c_uint,
                                      vp, sz, ctypes.c_int, ctypes.POINTER(ArPlan)]
    lib.ar_plan_query_add.restype = ctypes.c_int
    lib.ar_reduce_rows.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_int, ctypes.POINTER(ArRows),
                                   ctypes.c_int, ctypes.c_int, ctypes.c_uint, vp, vp]
    lib.ar_reduce_rows.restype = ctypes.c_int
    lib.ar_plan_query_rows.argtypes = [ctypes.POINTER(ArConfig), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                       ctypes.c_int, ctypes.POINTER(ArRows), ctypes.c_int, ctypes.c_int,
                                       ctypes.c_uint, vp, ctypes.c_int, ctypes.POINTER(ArPlan)]
    lib.ar_plan_query_rows.restype = ctypes.c_int
    lib.ar_qk_norm_rope.argtypes = [vp, ctypes.POINTER(ArQk), ctypes.c_int] + [vp] * 12
    lib.ar_attention.argtypes = [vp, ctypes.POINTER(ArAttn), ctypes.c_int] + [vp] * 9 + [sz, vp]
    lib.ar_attention_workspace.argtypes = [ctypes.POINTER(ArAttn), ctypes.c_int, ctypes.POINTER(sz)]
    lib.ar_fp8_quantize.argtypes = [vp] * 4 + [sz] * 4 + [ctypes.c_int, vp]
    lib.ar_fp8_matmul.argtypes = [vp, ctypes.POINTER(ArMm), ctypes.c_int] + [vp] * 6 + [sz, vp]
    lib.ar_fp8_matmul_workspace.argtypes = [ctypes.POINTER(ArMm), ctypes.c_int, ctypes.POINTER(sz)]
    for fn in (lib.ar_qk_norm_rope, lib.ar_attention, lib.ar_attention_workspace, lib.ar_fp8_quantize,
               lib.ar_fp8_matmul, lib.ar_fp8_matmul_workspace):
        fn.restype = ctypes.c_int
    _lib = lib
    return lib


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    raise TypeError(f"expected a tensor or an integer address, got {type(x).__name__}")


def ptr_array(xs):
    """A C array of pointers (``void *[]``) for dsts / srcs; build it once and
    reuse it across calls on the same buffers."""
    if xs is None:
        return None
    if isinstance(xs, ctypes.Array):
        return xs
    vals = [_addr(x) for x in xs]
    return (ctypes.c_void_p * max(1, len(vals)))(*vals)


_ptr_array = ptr_array

_TYPE_BYTES = {AR_F32: 4, AR_F16: 2, AR_BF16: 2}


def _tensors(xs):
    """The tensor entries of a dsts / srcs argument (addresses, None and
    ready-made pointer arrays are not checkable)."""
    if xs is None or isinstance(xs, ctypes.Array):
        return ()
    return [x for x in xs if x is not None and not isinstance(x, int)]


def _check_flat(xs, need: int, what: str) -> None:
    """1-D calls: each tensor is contiguous and holds at least ``need`` bytes."""
    for x in _tensors(xs):
        if x.nbytes < need or not x.is_contiguous():
            raise ValueError(f"{what}: a tensor of {x.nbytes} bytes{'' if x.is_contiguous() else ' (not contiguous)'}"
                             f" where the call reads or writes {need} contiguous bytes")


def _check_span(xs, need: int, what: str) -> None:
    """Row-strided calls: each tensor's storage holds ``need`` bytes from its data pointer."""
    for x in _tensors(xs):
        have = x.untyped_storage().nbytes() - x.storage_offset() * x.element_size()
        if have < need:
            raise ValueError(f"{what}: {have} bytes from the tensor's data pointer where the call spans {need}")


def _check_counts(dsts, srcs, mode: int, R: int | None = None) -> None:
    """The library reads R source pointers and n_dst destination pointers (n_dst = R
    for AR_MODE_RS_BCAST, else 1) from the arrays it is given: refuse lists shorter
    than that before building them (ctypes arrays and raw addresses are passed
    through as given, as in C).  Counts outside 2..AR_MAX_RANKS are left to the
    library, which rejects them before reading any pointer."""
    R = (len(srcs) if srcs is not None and not isinstance(srcs, ctypes.Array) else None) if R is None else R
    if R is None or not 2 <= R <= AR_MAX_RANKS:
        return
    if srcs is not None and not isinstance(srcs, ctypes.Array) and len(srcs) < R:
        raise ValueError(f"srcs has {len(srcs)} entries for R = {R}")
    n_dst = R if (int(mode) & AR_MODE_MASK) == AR_MODE_RS_BCAST else 1
    if dsts is not None and not isinstance(dsts, ctypes.Array) and len(dsts) < n_dst:
        raise ValueError(f"dsts has {len(dsts)} entries; this mode writes {n_dst} destinations")


def _flat_arrays(dsts, srcs, n: int, dst_type: int, wire_type: int, mode: int, validate: bool):
    """ptr_array(dsts), ptr_array(srcs) of a 1-D call, checking each tensor on the
    way (one pass: the check costs little beyond the pointer conversion); returns
    the arrays and the element width of the destination type (0 when unchecked)."""
    _check_counts(dsts, srcs, mode)
    dst_b = src_b = 0
    if validate and n > 0:
        dst_b = _TYPE_BYTES.get(dst_type, 0)
        src_b = _TYPE_BYTES.get(wire_type if mode & AR_SRC_WIRE else dst_type, 0)
        if not dst_b or not src_b:              # the library rejects the call itself
            dst_b = src_b = 0
    return _checked_array(dsts, n * dst_b, "dsts"), _checked_array(srcs, n * src_b, "srcs"), dst_b


def _checked_array(xs, need: int, what: str):
    """ptr_array(xs); with ``need`` > 0 every tensor must be contiguous and hold that many bytes."""
    if xs is None or isinstance(xs, ctypes.Array):
        return xs
    vals = []
    for x in xs:
        if x is None or isinstance(x, int):
            vals.append(x)
            continue
        vals.append(_addr(x))
        if need and (x.nbytes < need or not x.is_contiguous()):
            _check_flat((x,), need, what)
    return (ctypes.c_void_p * max(1, len(vals)))(*vals)


def _validate_rows(dsts, srcs, rows: int, cols: int, src_stride: int, dst_stride: int, dst_type: int,
                   wire_type: int, mode: int, residual, res_stride: int) -> None:
    dst_b = _TYPE_BYTES.get(int(dst_type))
    src_b = _TYPE_BYTES.get(int(wire_type) if int(mode) & AR_SRC_WIRE else int(dst_type))
    if dst_b is None or src_b is None or int(rows) <= 0 or int(cols) <= 0:
        return

    def extent(stride):
        return ((int(rows) - 1) * int(stride) + int(cols)) if int(stride) > 0 else int(cols)
    _check_span(dsts, extent(dst_stride) * dst_b, "dsts")
    _check_span(srcs, extent(src_stride) * src_b, "srcs")
    if residual is not None:
        _check_span((residual,), extent(res_stride) * dst_b, "residual")


def _stream_handle(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _config(config) -> ArConfig | None:
    if config is None:
        return None
    if isinstance(config, ArConfig):
        return config
    return ArConfig(**config)


def ar_status_str(status: int) -> str:
    return load_library().ar_status_str(int(status)).decode()


def ar_init(device: int = 0, config=None) -> ctypes.c_void_p:
    """Create a reduce context on HIP device ``device`` (raises ArError)."""
    lib = load_library()
    out = ctypes.c_void_p()
    cfg = _config(config)
    rc = lib.ar_init(ctypes.byref(out), int(device), ctypes.byref(cfg) if cfg is not None else None)
    if rc != AR_OK:
        raise ArError(rc, "ar_init")
    return out


def ar_reduce(ctx, dsts, srcs, n: int, dst_type: int = AR_F32, wire_type: int = AR_BF16,
              mode: int = AR_MODE_AUTO, stream=None, check: bool = True, validate: bool = True) -> int:
    """Enqueue one reduce; returns the status (raises ArError on failure if
    ``check``; ValueError before the call if ``validate`` finds a tensor too small)."""
    lib = load_library()
    n, dst_type, wire_type, mode = int(n), int(dst_type), int(wire_type), int(mode)
    dst_arr, src_arr, _ = _flat_arrays(dsts, srcs, n, dst_type, wire_type, mode, validate)
    R = len(srcs) if srcs is not None else 0
    rc = lib.ar_reduce(ctx, dst_arr, src_arr, R, n, dst_type, wire_type, mode, _stream_handle(stream))
    if check and rc != AR_OK:
        raise ArError(rc, "ar_reduce")
    return rc


def ar_reduce_staged_static(ctx, dsts, srcs, n: int, dst_type: int = AR_F32, wire_type: int = AR_BF16,
                            mode: int = AR_MODE_HOST_STAGED, stream=None, check: bool = True,
                            validate: bool = True) -> int:
    """The host-staged reduce with its staging ring in the library's static device
    array (no device allocation); arguments and checks as ar_reduce."""
    lib = load_library()
    n, dst_type, wire_type, mode = int(n), int(dst_type), int(wire_type), int(mode)
    dst_arr, src_arr, _ = _flat_arrays(dsts, srcs, n, dst_type, wire_type, mode, validate)
    R = len(srcs) if srcs is not None else 0
    rc = lib.ar_reduce_staged_static(ctx, dst_arr, src_arr, R, n, dst_type, wire_type, mode, _stream_handle(stream))
    if check and rc != AR_OK:
        raise ArError(rc, "ar_reduce_staged_static")
    return rc


def bind_reduce(ctx, dsts, srcs, n: int, dst_type: int = AR_F32, wire_type: int = AR_BF16,
                mode: int = AR_MODE_AUTO, stream=None, residual=None, residual_len: int | None = None):
    """One reduce with every argument converted to its C type once: returns a
    callable that enqueues the call again each time it is invoked and returns
    the status (no Python-side checks per call; the library still validates
    every call).  For latency-bound callers that issue the same call shape on
    the same buffers many times.  With ``residual`` it binds ``ar_reduce_add``.
    The caller keeps the context and the bound buffers alive while the callable is in use."""
    import functools

    lib = load_library()
    R = len(srcs)
    ctx_val = ctx.value if isinstance(ctx, ctypes.c_void_p) else ctx
    st_val = _stream_handle(stream)
    rlen = int(n) if residual_len is None else int(residual_len)
    if residual is not None and residual_len is None and hasattr(residual, "numel"):
        rlen = int(residual.numel())
    dst_arr, src_arr, dst_b = _flat_arrays(dsts, srcs, int(n), int(dst_type), int(wire_type), int(mode), True)
    if residual is not None and dst_b:
        _check_flat((residual,), rlen * dst_b, "residual")
    fast = _fast_module()
    if fast is not None:
        fn = lib.ar_reduce if residual is None else lib.ar_reduce_add
        return fast.bind(ctypes.cast(fn, ctypes.c_void_p).value, residual is not None, ctx_val or 0,
                         ctypes.addressof(dst_arr), ctypes.addressof(src_arr), R, int(n), int(dst_type),
                         int(wire_type), int(mode), _addr(residual) or 0, rlen, st_val or 0,
                         (dst_arr, src_arr))
    head = (ctypes.c_void_p(ctx_val), dst_arr, src_arr, ctypes.c_int(R), ctypes.c_size_t(int(n)),
            ctypes.c_int(int(dst_type)), ctypes.c_int(int(wire_type)), ctypes.c_uint(int(mode)))
    st = ctypes.c_void_p(st_val)
    if residual is None:
        return functools.partial(lib.ar_reduce, *head, st)
    return functools.partial(lib.ar_reduce_add, *head, ctypes.c_void_p(_addr(residual)), ctypes.c_size_t(rlen), st)


_fast = None


def _fast_module():
    """The compiled fast-call type (csrc/ar_pycall.c), or None when it was not built."""
    global _fast
    if _fast is None:
        try:
            from . import _ar_fast
            _fast = _ar_fast
        except ImportError:
            _fast = False
    return _fast or None


def ar_reduce_add(ctx, dsts, srcs, n: int, dst_type: int, wire_type: int, mode: int, residual,
                  residual_len: int | None = None, stream=None, check: bool = True,
                  validate: bool = True) -> int:
    """Enqueue one reduce followed by a residual add (element-wise when
    ``residual_len == n``, else one broadcast row); ``residual_len`` defaults to
    the residual tensor's element count.  Returns the status (raises ArError on
    failure if ``check``; ValueError before the call if ``validate`` finds a tensor too small)."""
    lib = load_library()
    R = len(srcs) if srcs is not None else 0
    if residual_len is None:
        if not hasattr(residual, "numel"):
            raise TypeError("residual_len is required when the residual is given as an address")
        residual_len = residual.numel()
    dst_arr, src_arr, dst_b = _flat_arrays(dsts, srcs, int(n), int(dst_type), int(wire_type), int(mode), validate)
    if dst_b:
        _check_flat((residual,), int(residual_len) * dst_b, "residual")
    rc = lib.ar_reduce_add(ctx, dst_arr, src_arr, R, int(n), int(dst_type),
                           int(wire_type), int(mode), _addr(residual), int(residual_len),
                           _stream_handle(stream))
    if check and rc != AR_OK:
        raise ArError(rc, "ar_reduce_add")
    return rc


def ar_reduce_rows(ctx, dsts, srcs, rows: int, cols: int, src_stride: int, dst_stride: int, dst_type: int,
                   wire_type: int, mode: int, residual=None, res_stride: int = 0, stream=None,
                   check: bool = True, validate: bool = True) -> int:
    """Enqueue one reduce of row-strided tensors (strides in elements); ``residual``
    None, or a tensor / address laid out with row stride ``res_stride`` (0 = one row
    added to every row).  Returns the status (raises ArError on failure if ``check``;
    ValueError before the call if ``validate`` finds a tensor's storage too small)."""
    lib = load_library()
    R = len(srcs) if srcs is not None else 0
    _check_counts(dsts, srcs, mode)
    if validate:
        _validate_rows(dsts, srcs, rows, cols, src_stride, dst_stride, dst_type, wire_type, mode, residual,
                       res_stride)
    shape = ArRows(int(rows), int(cols), int(src_stride), int(dst_stride), int(res_stride))
    rc = lib.ar_reduce_rows(ctx, _ptr_array(dsts), _ptr_array(srcs), R, ctypes.byref(shape), int(dst_type),
                            int(wire_type), int(mode), _addr(residual), _stream_handle(stream))
    if check and rc != AR_OK:
        raise ArError(rc, "ar_reduce_rows")
    return rc


def bind_reduce_rows(ctx, dsts, srcs, rows: int, cols: int, src_stride: int, dst_stride: int, dst_type: int,
                     wire_type: int, mode: int, residual=None, res_stride: int = 0, stream=None):
    """ar_reduce_rows with every argument converted to its C type once (the tensors'
    spans checked once, as ar_reduce_rows checks them): returns a callable that
    enqueues the call again each time it is invoked and returns the status (the
    library still validates every call).  The caller keeps the context and the
    bound buffers alive while the callable is in use."""
    import functools

    lib = load_library()
    R = len(srcs) if srcs is not None else 0
    _check_counts(dsts, srcs, mode)
    _validate_rows(dsts, srcs, rows, cols, src_stride, dst_stride, dst_type, wire_type, mode, residual, res_stride)
    shape = ctypes.pointer(ArRows(int(rows), int(cols), int(src_stride), int(dst_stride), int(res_stride)))
    ctx_val = ctx.value if isinstance(ctx, ctypes.c_void_p) else ctx
    return functools.partial(lib.ar_reduce_rows, ctypes.c_void_p(ctx_val), _ptr_array(dsts), _ptr_array(srcs),
                             ctypes.c_int(R), shape, ctypes.c_int(int(dst_type)), ctypes.c_int(int(wire_type)),
                             ctypes.c_uint(int(mode)), ctypes.c_void_p(_addr(residual)),
                             ctypes.c_void_p(_stream_handle(stream)))


# ---------------------------------------------------------------- layer operators

def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _type_code(x, what: str) -> int:
    code = {"torch.float32": AR_F32, "torch.float16": AR_F16, "torch.bfloat16": AR_BF16}.get(str(x.dtype))
    _need(code is not None, f"{what}: {x.dtype} is not float32, float16 or bfloat16")
    return code


# What a call's tensors are checked for and the C structure made of them depend on
# their sizes, strides and types alone: checked once for each such layout.
# Only the layouts are kept, no tensor and no address; a structure is copied where a call
# changes it.  Memory that is not on the context's device the library refuses; what it
# refuses is looked at again for tensors of several devices.
_layouts: dict = {}


def _layout(kind, tensors, extra, make):
    key = (kind, extra, *[None if x is None else (x.shape, x.stride(), x.dtype) for x in tensors])
    found = _layouts.get(key)
    if found is None:
        found = make()
        if len(_layouts) >= 4096:
            _layouts.clear()
        _layouts[key] = found
    return found


def _heads(x, what: str, like=None):
    """(token stride, head stride) of a [tokens, heads, head_dim] tensor.  A dimension of
    one element has no stride of its own: torch may report any for it."""
    _need(x.dim() == 3 and (x.shape[2] == 1 or x.stride(2) == 1),
          f"{what}: expected [tokens, heads, head_dim] with contiguous head_dim")
    if like is not None:
        _need(x.dtype == like.dtype and x.shape[2] == like.shape[2], f"{what}: type or head_dim differs from q's")
    dim = x.shape[2]
    return x.stride(0) if x.shape[0] > 1 else dim, x.stride(1) if x.shape[1] > 1 else dim


def _index(x, n: int, dtype: str, what: str) -> None:
    _need(str(x.dtype) == dtype and x.dim() == 1 and x.is_contiguous() and x.numel() == n,
          f"{what}: expected {n} contiguous {dtype} values")


def _flat_f32(x, n: int, what: str) -> None:
    _need(str(x.dtype) == "torch.float32" and x.is_contiguous() and x.numel() == n,
          f"{what}: expected {n} contiguous float32 values")


def _status(rc: int, what: str, check: bool, tensors=()) -> int:
    if rc == AR_ERR_INVALID:
        _need(len({x.get_device() for x in tensors if x is not None}) < 2, "tensors of one call live on one device")
    if check and rc != AR_OK:
        raise ArError(rc, what)
    return rc


def _ptr(x):
    return None if x is None else x.data_ptr()


def _call_stream(stream, like) -> int | None:
    """The handle of a layer operator's stream: torch's current one unless another is given.  (Its
    handle is asked for without making a stream object of it, which takes 2 of a single token's 10 us.)"""
    if stream is not None or not like.is_cuda:
        return _stream_handle(stream)
    import torch

    return torch._C._cuda_getCurrentRawStream(like.get_device())


def _workspace(need: int, given, like, stream, handle):
    """``given``, or bytes from torch's allocator for the stream of the call (so that
    they are not handed out again before the call's work there is done)."""
    if need == 0:
        return None
    if given is not None:
        _need(given.is_contiguous(), "workspace: expected contiguous bytes")
        return given
    import torch

    handle = handle or 0
    if stream is None or torch.cuda.current_stream(like.device).cuda_stream == handle:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    on = torch.cuda.ExternalStream(handle, like.device) if handle else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(on):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def _qk_layout(q, k, q_weight, k_weight, table, positions, q_out, k_out, v, v_out, slots):
    s = ArQk()
    s.q_token, s.q_head = _heads(q, "q")
    s.k_token, s.k_head = _heads(k, "k", q)
    s.q_out_token, s.q_out_head = _heads(q_out, "q_out", q)
    s.k_out_token, s.k_out_head = _heads(k_out, "k_out", q)
    s.tokens, s.heads_q, s.head_dim = tokens, _, dim = tuple(q.shape)
    s.heads_kv = k.shape[1]
    _need(q_out.shape == q.shape and k.shape[0] == tokens and k_out.shape[1] == k.shape[1], "sizes of q, k and outputs differ")
    if v is not None:
        s.v_token, s.v_head = _heads(v, "v", q)
        s.v_out_token, s.v_out_head = _heads(v_out, "v_out", q)
        _need(v.shape == k.shape and v_out.shape == k_out.shape, "sizes of v and v_out differ from k's and k_out's")
    if slots is None:
        _need(k_out.shape[0] == tokens, "without slots k_out has a row for each token")
    else:
        _index(slots, tokens, "torch.int64", "slots")
        s.cache_rows = k_out.shape[0]
    for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        _need(w is None or (w.dtype == q.dtype and w.is_contiguous() and w.numel() == dim),
              f"{what}: expected head_dim contiguous values of q's type")
    if table is not None:
        _need(str(table.dtype) == "torch.float32" and table.dim() == 2 and table.is_contiguous() and positions is not None,
              "table: expected contiguous float32 [positions, rot_dim], and positions")
        s.table_rows, s.rot_dim = table.shape
        _index(positions, tokens, "torch.int64", "positions")
    return s, _type_code(q, "q")


def ar_qk_norm_rope(ctx, q, k, q_weight=None, k_weight=None, table=None, positions=None, q_out=None, k_out=None,
                    v=None, v_out=None, slots=None, eps: float = 1e-6, interleaved: bool = False, stream=None,
                    check: bool = True) -> int:
    """Norm of each head's queries and keys and the position rotation in one pass.

    ``q`` [tokens, heads_q, head_dim], ``k`` [tokens, heads_kv, head_dim] (any token and head
    strides); ``q_weight`` / ``k_weight`` [head_dim] or None; ``table`` [positions, rot_dim] float32,
    a position's cosines and then its sines (None: no rotation); ``positions`` [tokens] int64.
    ``q_out`` / ``k_out`` default to in place.  With ``slots`` [tokens] int64 the keys (and
    ``v`` into ``v_out``) go to those rows of ``k_out`` [cache_rows, heads_kv, head_dim]; a slot
    outside it (-1) writes neither.  Returns the status (raises ArError if ``check``)."""
    lib = load_library()
    if q_out is None:
        q_out = q
    if k_out is None:
        _need(slots is None, "slots need a k_out")
        k_out = k
    _need((v is None) == (v_out is None), "v and v_out come together")
    tensors = (q, k, q_weight, k_weight, table, positions, q_out, k_out, v, v_out, slots)

    def make():
        s, code = _qk_layout(*tensors)
        s.eps = eps
        s.flags = AR_QK_INTERLEAVED if interleaved else 0
        return ctypes.pointer(s), code
    shape, code = _layout("qk", tensors, (eps, interleaved), make)
    rc = lib.ar_qk_norm_rope(ctx, shape, code, q_out.data_ptr(), k_out.data_ptr(), _ptr(v_out), q.data_ptr(), k.data_ptr(),
                             _ptr(v), _ptr(q_weight), _ptr(k_weight), _ptr(table),
                             None if table is None else positions.data_ptr(), _ptr(slots), _call_stream(stream, q))
    return _status(rc, "ar_qk_norm_rope", check, tensors)


def _attn_layout(out, q, k, v) -> ArAttn:
    s = ArAttn()
    s.q_token, s.q_head = _heads(q, "q")
    s.k_token, s.k_head = _heads(k, "k", q)
    s.v_token, s.v_head = _heads(v, "v", q)
    s.o_token, s.o_head = _heads(out, "out", q)
    s.total_q, s.heads_q, s.head_dim = q.shape
    s.rows_k, s.heads_kv, _ = k.shape
    _need(out.shape == q.shape and v.shape == k.shape, "out has q's sizes and v has k's")
    return s


def _attn_call(s: ArAttn, batch: int, max_q: int, max_k: int, causal: bool, scale) -> ArAttn:
    s = ArAttn.from_buffer_copy(s)
    # (an assignment to a C int drops what does not fit into it)
    s.batch, s.max_q, s.max_k = batch, *(max(-1, min(int(x), (1 << 31) - 1)) for x in (max_q, max_k))
    s.scale = s.head_dim ** -0.5 if scale is None else float(scale)
    s.flags = AR_ATTN_CAUSAL if causal else 0
    return s


def ar_attention_workspace(out, q, k, v, batch: int, max_q: int, max_k: int, causal: bool = True, scale=None) -> int:
    """Bytes of workspace that ar_attention needs for these tensors."""
    s, need = _attn_call(_attn_layout(out, q, k, v), batch, max_q, max_k, causal, scale), ctypes.c_size_t()
    _status(load_library().ar_attention_workspace(ctypes.byref(s), _type_code(q, "q"), ctypes.byref(need)),
            "ar_attention_workspace", True)
    return need.value


def ar_attention(ctx, out, q, k, v, cu_q, k_start, k_len, max_q: int, max_k: int, causal: bool = True, scale=None,
                 lse=None, workspace=None, stream=None, check: bool = True) -> int:
    """Attention of packed sequences over a prompt or a cache.

    ``q`` / ``out`` [total_q, heads_q, head_dim]; ``k`` / ``v`` [rows, heads_kv, head_dim] (any
    token and head strides).  Sequence b's queries are rows ``cu_q[b]`` .. ``cu_q[b + 1]`` (int32), its
    keys rows ``k_start[b]`` (int64) .. + ``k_len[b]`` (int32); ``max_q`` / ``max_k`` bound the lengths.
    ``causal``: the last query sees every key, each earlier one a key less.  ``scale`` defaults to
    head_dim ** -0.5.  ``lse`` [total_q, heads_q] float32 is optional.  ``workspace`` (uint8,
    ar_attention_workspace bytes) defaults to torch's allocator.  Returns the status."""
    lib = load_library()

    def make():
        s = _attn_layout(out, q, k, v)
        batch = k_len.numel()
        _index(cu_q, batch + 1, "torch.int32", "cu_q")
        _index(k_start, batch, "torch.int64", "k_start")
        _index(k_len, batch, "torch.int32", "k_len")
        if lse is not None:
            _flat_f32(lse, s.total_q * s.heads_q, "lse")
        return s, _type_code(q, "q"), batch
    tensors = (out, q, k, v, cu_q, k_start, k_len, lse)
    layout, code, batch = _layout("attn", tensors, None, make)
    s = _attn_call(layout, batch, max_q, max_k, causal, scale)
    need = ctypes.c_size_t()
    rc = lib.ar_attention_workspace(ctypes.byref(s), code, ctypes.byref(need))
    if rc == AR_OK:
        handle = _call_stream(stream, q)
        ws = _workspace(need.value, workspace, q, stream, handle)
        rc = lib.ar_attention(ctx, ctypes.byref(s), code, out.data_ptr(), _ptr(lse), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                              cu_q.data_ptr(), k_start.data_ptr(), k_len.data_ptr(), _ptr(ws),
                              0 if ws is None else ws.nbytes, handle)
    return _status(rc, "ar_attention", check, tensors)


def _codes(x, what: str) -> int:
    _need(str(x.dtype) in ("torch.float8_e4m3fn", "torch.uint8") and x.dim() == 2 and (x.shape[1] <= 1 or x.stride(1) == 1),
          f"{what}: expected a row-major matrix of float8_e4m3fn (or uint8) codes")
    return _row(x, 16)


def _row(x, step: int) -> int:
    """A matrix's row stride; a single or an empty row has none of its own, so the next multiple of ``step``."""
    return x.stride(0) if x.shape[0] > 1 and x.shape[1] > 0 else -(-x.shape[1] // step) * step


def ar_fp8_quantize(ctx, codes, scales, x, stream=None, check: bool = True) -> int:
    """e4m3 codes [rows, cols] of ``x`` [rows, cols] with a float32 scale for each block of 128
    elements of a row (``scales`` [rows, ceil(cols / 128)]).  Returns the status."""
    lib = load_library()

    def make():
        _need(x.dim() == 2 and (x.shape[1] <= 1 or x.stride(1) == 1) and codes.shape == x.shape,
              "x: expected a row-major matrix, and codes of its sizes")
        rows, cols = x.shape
        codes_row = _codes(codes, "codes")
        _flat_f32(scales, rows * -(-cols // AR_F8_BLOCK), "scales")
        return rows, cols, _row(x, 8), codes_row, _type_code(x, "x")
    tensors = (codes, scales, x)
    sizes = _layout("quant", tensors, None, make)
    rc = lib.ar_fp8_quantize(ctx, codes.data_ptr(), scales.data_ptr(), x.data_ptr(), *sizes, _call_stream(stream, x))
    return _status(rc, "ar_fp8_quantize", check, tensors)


def _mm_layout(out, a, b) -> ArMm:
    _need(out.dim() == 2 and (out.shape[1] <= 1 or out.stride(1) == 1), "out: expected a row-major matrix")
    s = ArMm(a.shape[0], b.shape[0], a.shape[1], _codes(a, "a"), _codes(b, "b"), _row(out, 1))
    _need(b.shape[1] == a.shape[1] and tuple(out.shape) == (a.shape[0], b.shape[0]),
          "sizes: out [rows, cols], a [rows, depth], b [cols, depth]")
    return s


def ar_fp8_matmul_workspace(out, a, b) -> int:
    """Bytes of workspace that ar_fp8_matmul needs for these tensors."""
    s, need = _mm_layout(out, a, b), ctypes.c_size_t()
    _status(load_library().ar_fp8_matmul_workspace(ctypes.byref(s), _type_code(out, "out"), ctypes.byref(need)),
            "ar_fp8_matmul_workspace", True)
    return need.value


def ar_fp8_matmul(ctx, out, a, a_scales, b, b_scales, workspace=None, stream=None, check: bool = True) -> int:
    """``out`` [rows, cols] = a b^T of e4m3 matrices ``a`` [rows, depth] and ``b`` [cols, depth] with
    float32 block scales ``a_scales`` [rows, ceil(depth / 128)] and ``b_scales`` [ceil(cols / 128),
    ceil(depth / 128)]; ``out`` in float32, or rounded once to a 16-bit wire type (a source for
    ar_reduce with AR_SRC_WIRE).  ``workspace`` (uint8) defaults to torch's allocator.  Returns the status."""
    lib = load_library()

    def make():
        s, need = _mm_layout(out, a, b), ctypes.c_size_t()
        code = _type_code(out, "out")
        blocks = -(-s.depth // AR_F8_BLOCK)
        _flat_f32(a_scales, s.rows * blocks, "a_scales")
        _flat_f32(b_scales, -(-s.cols // AR_F8_BLOCK) * blocks, "b_scales")
        rc = lib.ar_fp8_matmul_workspace(ctypes.byref(s), code, ctypes.byref(need))
        return ctypes.pointer(s), code, need.value, rc
    tensors = (out, a, a_scales, b, b_scales)
    shape, code, need, rc = _layout("mm", tensors, None, make)
    if rc == AR_OK:
        handle = _call_stream(stream, out)
        ws = _workspace(need, workspace, out, stream, handle)
        rc = lib.ar_fp8_matmul(ctx, shape, code, out.data_ptr(), a.data_ptr(), a_scales.data_ptr(), b.data_ptr(),
                               b_scales.data_ptr(), _ptr(ws), 0 if ws is None else ws.nbytes, handle)
    return _status(rc, "ar_fp8_matmul", check, tensors)


def ar_free(ctx) -> None:
    rc = load_library().ar_free(ctx)
    if rc != AR_OK:
        raise ArError(rc, "ar_free")


def ar_plan_query(dsts, srcs, n: int, dst_type: int = AR_F32, wire_type: int = AR_BF16,
                  mode: int = AR_MODE_AUTO, srcs_on_host: bool = False, config=None,
                  R: int | None = None):
    """Host-only validation + plan; returns (status, ArPlan)."""
    lib = load_library()
    plan = ArPlan()
    cfg = _config(config)
    R = (len(srcs) if srcs is not None else 0) if R is None else R
    _check_counts(dsts, srcs, mode, R)
    rc = lib.ar_plan_query(ctypes.byref(cfg) if cfg is not None else None, _ptr_array(dsts),
                           _ptr_array(srcs), R, int(n), int(dst_type), int(wire_type), int(mode),
                           int(bool(srcs_on_host)), ctypes.byref(plan))
    return rc, plan


def ar_plan_query_add(dsts, srcs, n: int, dst_type: int, wire_type: int, mode: int, residual,
                      residual_len: int, srcs_on_host: bool = False, config=None, R: int | None = None):
    """Host-only validation + plan of ar_reduce_add; returns (status, ArPlan)."""
    lib = load_library()
    plan = ArPlan()
    cfg = _config(config)
    R = (len(srcs) if srcs is not None else 0) if R is None else R
    _check_counts(dsts, srcs, mode, R)
    rc = lib.ar_plan_query_add(ctypes.byref(cfg) if cfg is not None else None, _ptr_array(dsts),
                               _ptr_array(srcs), R, int(n), int(dst_type), int(wire_type), int(mode),
                               _addr(residual), int(residual_len), int(bool(srcs_on_host)),
                               ctypes.byref(plan))
    return rc, plan


def ar_plan_query_rows(dsts, srcs, rows: int, cols: int, src_stride: int, dst_stride: int, dst_type: int,
                       wire_type: int, mode: int, residual=None, res_stride: int = 0, srcs_on_host: bool = False,
                       config=None, R: int | None = None):
    """Host-only validation + plan of ar_reduce_rows; returns (status, ArPlan)."""
    lib = load_library()
    plan = ArPlan()
    cfg = _config(config)
    R = (len(srcs) if srcs is not None else 0) if R is None else R
    _check_counts(dsts, srcs, mode, R)
    shape = ArRows(int(rows), int(cols), int(src_stride), int(dst_stride), int(res_stride))
    rc = lib.ar_plan_query_rows(ctypes.byref(cfg) if cfg is not None else None, _ptr_array(dsts),
                                _ptr_array(srcs), R, ctypes.byref(shape), int(dst_type), int(wire_type),
                                int(mode), _addr(residual), int(bool(srcs_on_host)), ctypes.byref(plan))
    return rc, plan


class Reducer:
    """Owns one context; ``reducer(dsts, srcs, ...)`` enqueues a reduce."""

    def __init__(self, device: int = 0, config=None):
        self.ctx = ar_init(device, config)

    def __call__(self, dsts, srcs, n=None, dst_type=AR_F32, wire_type=AR_BF16,
                 mode=AR_MODE_AUTO, stream=None):
        if n is None:
            first = next((s for s in srcs if s is not None), None)
            if first is None:
                raise ValueError("n is required when every source is inactive")
            n = first.numel()
        return ar_reduce(self.ctx, dsts, srcs, n, dst_type, wire_type, mode, stream)

    def close(self):
        if self.ctx is not None:
            ar_free(self.ctx)
            self.ctx = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
