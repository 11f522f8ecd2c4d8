"""ctypes binding over the C ABI in ``include/`` (``mbrs_softmax.h``,
``mbrs_attention.h``, ``mbrs_sequence.h``).

Argument marshalling only: every step of the softmax runs in the CUDA kernels
of ``_build/libmbrs_softmax.so``.  If that library has not been built, the
first call raises -- there is no other implementation to fall back to.
PyTorch supplies device memory and the current stream.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libmbrs_softmax.so")

OK, ERR_NULL, ERR_SHAPE, ERR_STRIDE, ERR_DTYPE, ERR_OVERLAP, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_ALIGN, \
    ERR_ARG, ERR_SCRATCH_LIMIT = range(12)
PATH_AUTO, PATH_WARP, PATH_CTA, PATH_CLUSTER, PATH_SPLIT = range(5)  # PATH_SPLIT: softmax_fwd_noalloc only
PATH_STREAM, PATH_PACKED, PATH_GRID = 6, 7, 8
PATH_NAMES = {PATH_WARP: "warp", PATH_CTA: "cta", PATH_CLUSTER: "cluster", PATH_SPLIT: "split",
              PATH_STREAM: "stream", PATH_PACKED: "packed", PATH_GRID: "grid"}
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}

_i64, _u64, _int, _vp = ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_void_p


class Plan(ctypes.Structure):
    _fields_ = [("path", _int), ("threads", _int), ("vpt", _int), ("group", _int), ("launches", _int),
                ("vec_store", _int), ("grid", _i64), ("smem_bytes", _i64), ("scratch_bytes", _i64),
                ("hbm_bytes", _i64), ("whole_vectors", _int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class TuneResult(ctypes.Structure):
    _fields_ = [("plan", Plan), ("best_us", ctypes.c_double), ("auto_us", ctypes.c_double), ("candidates", _int)]


class AttentionPlan(ctypes.Structure):
    _fields_ = [("items", _i64), ("grid", _i64), ("head_group", _int), ("threads", _int), ("smem_bytes", _i64),
                ("tmem_columns", _int), ("flops", ctypes.c_double)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class SequenceArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("q", "k", "v", "o", "lse", "q_starts", "kv_lens", "page_table")] + \
               [(n, _i64) for n in ("q_token_stride", "q_head_stride", "k_page_stride", "k_token_stride", "k_head_stride",
                                    "v_page_stride", "v_token_stride", "v_head_stride", "o_token_stride",
                                    "o_head_stride", "table_stride", "tokens", "batch", "heads", "kv_heads", "head_dim",
                                    "pages", "page_size", "max_pages")] + \
               [("dtype", _int), ("causal", _int), ("sm_scale", ctypes.c_float)]


class AppendArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "k_cache", "v_cache", "q", "q_out", "q_starts", "kv_lens", "page_table",
                                   "inv_freq")] + \
               [(n, _i64) for n in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride",
                                    "q_token_stride", "q_head_stride", "q_out_token_stride", "q_out_head_stride",
                                    "k_cache_page_stride", "k_cache_token_stride", "k_cache_head_stride",
                                    "v_cache_page_stride", "v_cache_token_stride", "v_cache_head_stride",
                                    "table_stride", "tokens", "batch", "heads", "kv_heads", "head_dim", "pages",
                                    "page_size", "max_pages", "rotary_dim")] + \
               [("interleaved", _int), ("dtype", _int)]


class Shape(ctypes.Structure):
    _fields_ = [("path", _int), ("threads", _int), ("vpt", _int), ("group", _int)]

    def as_tuple(self) -> tuple:
        return (self.path, self.threads, self.vpt, self.group)


# Every function the header declares, with its ctypes signature.
SIGNATURES = {
    "softmax_fwd": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp]),
    "softmax_status_string": (ctypes.c_char_p, [_int]),
    "softmax_last_path": (_int, []),
    "softmax_set_force_path": (_int, [_int, _int, _int, _int]),
    "softmax_plan": (_int, [_u64, _u64, _i64, _i64, _i64, _int, _int, ctypes.POINTER(Plan)]),
    "softmax_check_device_error": (_int, [_vp]),
    "softmax_set_wait_test": (_int, [_i64, _int]),
    "softmax_set_launch_overlap": (_int, [_int]),
    "softmax_fwd_host": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp]),
    "softmax_host_workspace_bytes": (_i64, [_i64, _i64, _i64, _int, _i64]),
    "softmax_autotune": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp, _int, ctypes.POINTER(TuneResult)]),
    "softmax_tune_candidates": (_int, [_u64, _u64, _i64, _i64, _i64, _int, _int, ctypes.POINTER(Shape), _int]),
    "softmax_autotune_size": (_int, []),
    "softmax_autotune_clear": (_int, []),
    "softmax_abi_version": (_int, []),
    "softmax_fwd_noalloc": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp]),
    "softmax_fwd_masked": (_int, [_vp, _vp, _i64, _i64, _i64, _int, ctypes.c_float, _i64, _i64, _vp]),
    "softmax_masked_copy": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _i64, _i64, _int, _vp]),
    "softmax_attention_fwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, ctypes.c_float, _vp]),
    "softmax_attention_fwd_counter": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, ctypes.c_float,
                                             _vp, _vp]),
    "softmax_attention_set_wait_test": (_int, [_int]),
    "softmax_attention_plan": (_int, [_i64, _i64, _i64, _i64, _int, _int, _int, ctypes.POINTER(AttentionPlan)]),
    "softmax_attention_varlen_fwd": (_int, [_vp, _vp, _i64, _vp]),
    "softmax_attention_paged_fwd": (_int, [_vp, _vp, _i64, _vp]),
    "softmax_sequence_workspace_bytes": (_i64, [_vp]),
    "softmax_kv_cache_append": (_int, [_vp, _vp]),
}

_lib = None
_lock = threading.Lock()


class SoftmaxError(RuntimeError):
    def __init__(self, status: int, what: str = "softmax_fwd"):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"CUDA library {_LIB_PATH} is missing: build it with "
                    "`python -m memory_bound_row_softmax_gb300.build` (there is no fallback path)")
            handle = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().softmax_status_string(status).decode()


def _torch_dtype_code(t) -> int:
    import torch
    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if t.dtype not in codes:
        raise TypeError(f"softmax_fwd takes float32, float16 or bfloat16, not {t.dtype}")
    return codes[t.dtype]


def softmax_fwd_ptr(in_ptr: int, out_ptr: int, rows: int, cols: int, row_stride: int, dtype: int,
                    stream: int = 0) -> int:
    """Raw call: device addresses and sizes in, status out (no exception)."""
    return lib().softmax_fwd(in_ptr, out_ptr, rows, cols, row_stride, dtype, stream)


def softmax_fwd_noalloc_ptr(in_ptr: int, out_ptr: int, rows: int, cols: int, row_stride: int, dtype: int,
                            stream: int = 0) -> int:
    """Raw call of the entry point that allocates nothing (for callers that
    cannot allocate device memory; its scratch is a fixed array in the
    library).  Status out, no exception."""
    return lib().softmax_fwd_noalloc(in_ptr, out_ptr, rows, cols, row_stride, dtype, stream)


def softmax_fwd_masked_ptr(in_ptr: int, out_ptr: int, rows: int, cols: int, row_stride: int, dtype: int,
                           scale: float, causal_offset: int, rows_per_seq: int = 0, stream: int = 0) -> int:
    """Raw call of the scaled, causally masked softmax (status out)."""
    return lib().softmax_fwd_masked(in_ptr, out_ptr, rows, cols, row_stride, dtype, scale, causal_offset,
                                    rows_per_seq, stream)


def masked_copy_ptr(in_ptr: int, out_ptr: int, rows: int, cols: int, row_stride: int, dtype: int,
                    causal_offset: int, rows_per_seq: int = 0, threads: int = 0, stream: int = 0) -> int:
    """Raw call of the diagnostic softmax_masked_copy: the masked call's
    traffic (kept entries copied, the rest zeroed) with no arithmetic."""
    return lib().softmax_masked_copy(in_ptr, out_ptr, rows, cols, row_stride, dtype, causal_offset, rows_per_seq,
                                     threads, stream)


def _prepare(x, out, what: str):
    """Check a 2-D CUDA tensor (last dimension contiguous) and its output;
    returns (rows, cols, row_stride, dtype code, out)."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{what} needs a CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"{what} needs a 2-D tensor, got {tuple(x.shape)}")
    rows, cols = x.shape
    if cols > 1 and x.stride(1) != 1:
        raise ValueError("the last dimension must be contiguous (stride 1)")
    row_stride = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    code = _torch_dtype_code(x)
    if out is None:
        out = torch.empty_strided((rows, cols), (row_stride, 1), dtype=x.dtype, device=x.device)
    else:
        if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
            raise ValueError("out must match x in shape, dtype and device")
        o_stride = out.stride(0) if rows > 1 else row_stride
        if (cols > 1 and out.stride(1) != 1) or o_stride != row_stride:
            raise ValueError("out must have x's row stride")
    return rows, cols, row_stride, code, out


def _stream_handle(x, stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def softmax_fwd(x, out=None, stream=None):
    """Row softmax of a 2-D CUDA tensor (last dimension contiguous).

    ``out`` (optional) must have x's shape, dtype, device and row stride; it
    may be ``x`` itself.  Launches on ``stream`` (default: the current stream of
    x's device) and returns ``out``.
    """
    import torch
    rows, cols, row_stride, code, out = _prepare(x, out, "softmax_fwd")
    with torch.cuda.device(x.device):
        st = lib().softmax_fwd(x.data_ptr(), out.data_ptr(), rows, cols, row_stride, code, _stream_handle(x, stream))
    if st != OK:
        raise SoftmaxError(st)
    return out


def softmax_fwd_masked(x, scale: float = 1.0, causal_offset: int = 0, rows_per_seq: int = 0, out=None,
                       stream=None):
    """Softmax of scaled, causally masked rows: row r keeps the columns
    c <= (r mod rows_per_seq) + causal_offset (rows_per_seq 0: r itself), its
    scores are x * scale, masked outputs are 0 and masked inputs are never
    read.  Arguments otherwise as ``softmax_fwd``; returns ``out``."""
    import torch
    rows, cols, row_stride, code, out = _prepare(x, out, "softmax_fwd_masked")
    with torch.cuda.device(x.device):
        st = lib().softmax_fwd_masked(x.data_ptr(), out.data_ptr(), rows, cols, row_stride, code, float(scale),
                                      int(causal_offset), int(rows_per_seq), _stream_handle(x, stream))
    if st != OK:
        raise SoftmaxError(st, "softmax_fwd_masked")
    return out


def attention_fwd_ptr(q: int, k: int, v: int, o: int, batch: int, heads: int, n_ctx: int, head_dim: int,
                      dtype: int, causal: bool, sm_scale: float, stream: int = 0) -> int:
    """Raw call of the fused attention forward (status out)."""
    return lib().softmax_attention_fwd(q, k, v, o, batch, heads, n_ctx, head_dim, dtype, 1 if causal else 0,
                                       sm_scale, stream)


def attention_fwd_counter_ptr(q: int, k: int, v: int, o: int, batch: int, heads: int, n_ctx: int, head_dim: int,
                              dtype: int, causal: bool, sm_scale: float, counter: int, stream: int = 0) -> int:
    """Raw call of the fused attention forward with the caller's two work
    counters at device address ``counter`` (status out)."""
    return lib().softmax_attention_fwd_counter(q, k, v, o, batch, heads, n_ctx, head_dim, dtype,
                                               1 if causal else 0, sm_scale, counter, stream)


def attention_fwd(q, k, v, causal: bool = True, sm_scale: float | None = None, out=None, stream=None):
    """Fused attention forward O = softmax(Q K^T * sm_scale [causal]) V of
    [batch, heads, n_ctx, 128] contiguous fp16 / bf16 CUDA tensors (sm_scale
    defaults to 1 / sqrt(head_dim)); returns ``out``."""
    import torch
    for t in (q, k, v):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("attention_fwd needs CUDA tensors")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError("attention_fwd needs contiguous [batch, heads, n_ctx, head_dim] tensors")
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one shape and dtype")
    batch, heads, n_ctx, head_dim = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / float(head_dim) ** 0.5
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    with torch.cuda.device(q.device):
        st = attention_fwd_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), batch, heads, n_ctx,
                               head_dim, _torch_dtype_code(q), causal, float(sm_scale), _stream_handle(q, stream))
    if st != OK:
        raise SoftmaxError(st, "attention_fwd")
    return out


# The sequence calls below are short on the GPU (a decode step's append takes
# a few microseconds), so their marshalling asks each tensor for its shape and
# strides once and packs the argument structs with struct.pack: 25 us of Python
# per call became 9 (with the kept workspace below).
_SEQUENCE_PACK = struct.Struct("@8P19qiif4x")
_APPEND_PACK = struct.Struct("@10P24qii")
assert _SEQUENCE_PACK.size == ctypes.sizeof(SequenceArgs) and _APPEND_PACK.size == ctypes.sizeof(AppendArgs)
_CODES: dict = {}  # torch dtype -> code; filled on first use (torch is imported late)
_INDEX: list = []  # torch's int32, likewise


def _refuse_tensor(t, what: str, name: str, dims: int, dtype, device):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what}: {name} must be a CUDA tensor")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what}: {name} must have dtype {dtype} on {device}")
    if t.dim() != dims:
        raise ValueError(f"{what}: {name} must have {dims} dimensions, got {tuple(t.shape)}")
    raise ValueError(f"{what}: the last dimension of {name} must be contiguous (stride 1)")


def _operand(t, what: str, name: str, dims: int, dtype, device):
    """(address, shape, strides) of a CUDA tensor of this dtype and device with
    `dims` dimensions, the last one contiguous; anything else is refused."""
    try:
        shape, strides = t.shape, t.stride()
        ok = len(strides) == dims and (strides[-1] == 1 or shape[-1] <= 1) and t.dtype is dtype and t.device == device
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        _refuse_tensor(t, what, name, dims, dtype, device)
    return t.data_ptr(), shape, strides


def _first_operand(t, what: str, name: str):
    """The same for the tensor that sets dtype and device; also returns those and the dtype's code."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what}: {name} must be a CUDA tensor")
    if not _CODES:
        _INDEX.append(torch.int32)
        _CODES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} takes float16 or bfloat16, not {t.dtype}")
    return (*_operand(t, what, name, 3, t.dtype, t.device), t.dtype, t.device, code)


def _indices(t, what: str, name: str, dims: int, device):
    """(address, shape, strides) of an int32 index tensor, its last dimension contiguous."""
    try:
        shape, strides = t.shape, t.stride()
        ok = t.dtype is _INDEX[0] and t.device == device
    except (AttributeError, TypeError):
        ok = False
    if not ok:
        raise TypeError(f"{what}: {name} must be an int32 tensor on {device}")
    if len(strides) != dims or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{what}: {name} must have {dims} dimensions, the last one contiguous, got {tuple(shape)}")
    return t.data_ptr(), shape, strides


def _starts(q_starts, what, device):
    """Batch and address of the row offsets."""
    ptr, (n,), _ = _indices(q_starts, what, "q_starts", 1, device)
    if n < 1:
        raise ValueError(f"{what}: q_starts must hold batch + 1 offsets")
    return n - 1, ptr


def _tables(what, page_table, kv_lens, q_starts, device):
    """The index tensors of a paged call: batch, max_pages, table_stride and their addresses."""
    batch, starts_ptr = _starts(q_starts, what, device)
    lens_ptr, (n,), _ = _indices(kv_lens, what, "kv_lens", 1, device)
    table_ptr, (rows, max_pages), (stride, _) = _indices(page_table, what, "page_table", 2, device)
    if n != batch or rows != batch:
        raise ValueError(f"{what}: q_starts must hold batch + 1 offsets, kv_lens batch lengths and page_table batch rows")
    return batch, max_pages, (stride if batch > 1 else max(max_pages, stride)), starts_ptr, lens_ptr, table_ptr


def _new_tensor(shape, dtype, like, stream):
    """A new tensor beside `like` that the given stream may write at once: allocated in its
    pool where it is not the current one, and known to the current one too."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    device = like.device
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(s):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(device))
    return t


# A call's workspace is allocated and freed in 4 us, and 3 more go in what that
# puts out of the host's caches, a third of a short call: so each thread keeps one
# for each stream that its calls went to (they follow one another there, and each
# writes what it reads).  Not while a capture is on (a graph's replays would meet
# the stream's other calls), not for a stream passed in, not above this size.
_KEPT_BYTES = 64 << 20
_KEPT_STREAMS = 8
_kept = threading.local()


def _workspace_of(need, q, device, handle):
    """A workspace of at least `need` bytes for a call on the current stream."""
    import torch
    if need > _KEPT_BYTES or torch.cuda.is_current_stream_capturing():
        return _new_tensor((need,), torch.uint8, q, None)
    kept = _kept.__dict__
    key = device.index, handle
    ws = kept.get(key)
    if ws is None or ws.nbytes < need:
        if ws is None and len(kept) >= _KEPT_STREAMS:
            kept.clear()
        kept[key] = ws = _new_tensor((need,), torch.uint8, q, None)
    return ws


def _stream_of(device, stream):
    """The handle of `stream`, or of the device's current one (asked for without
    building a Stream object, 2 us a call, where torch offers that)."""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream


def _sequence_attention(what, call, q, k, v, paged, causal, sm_scale, q_starts, out, lse, workspace, stream):
    import torch
    q_ptr, (tokens, heads, head_dim), qs, dtype, device, code = _first_operand(q, what, "q")
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _sequence_attention(what, call, q, k, v, paged, causal, sm_scale, q_starts, out, lse, workspace, stream)
    if paged is None:
        k_ptr, ksh, ks = _operand(k, what, "k", 3, dtype, device)
        v_ptr, vsh, vs = _operand(v, what, "v", 3, dtype, device)
        if ksh != vsh or ksh[0] != tokens or ksh[2] != head_dim:
            raise ValueError(f"{what}: k and v must be [tokens, kv_heads, head_dim] of q's tokens and head_dim")
        batch, starts_ptr = _starts(q_starts, what, device)
        strides = (0, ks[0], ks[1], 0, vs[0], vs[1])
        lens_ptr = table_ptr = table_stride = pages = page_size = max_pages = 0
        kv_heads = ksh[1]
    else:
        k_ptr, ksh, ks = _operand(k, what, "k_cache", 4, dtype, device)
        v_ptr, vsh, vs = _operand(v, what, "v_cache", 4, dtype, device)
        if ksh != vsh or ksh[3] != head_dim:
            raise ValueError(f"{what}: k_cache and v_cache must have one shape and q's head_dim")
        batch, max_pages, table_stride, starts_ptr, lens_ptr, table_ptr = _tables(what, *paged, q_starts, device)
        strides = (*ks[:3], *vs[:3])
        pages, page_size, kv_heads = ksh[0], ksh[1], ksh[2]
    if sm_scale is None:
        sm_scale = 1.0 / float(head_dim) ** 0.5
    if out is None:
        out = _new_tensor((tokens, heads, head_dim), dtype, q, stream)
    o_ptr, osh, os_ = _operand(out, what, "out", 3, dtype, device)
    if osh != q.shape:
        raise ValueError(f"{what}: out must have q's shape")
    lse_ptr = 0
    if lse is not None:
        lse_ptr, lsh, _ = _operand(lse, what, "lse", 2, torch.float32, device)
        if lsh != (tokens, heads) or not lse.is_contiguous():
            raise ValueError(f"{what}: lse must be a contiguous [tokens, heads] tensor")
    args = _SEQUENCE_PACK.pack(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, starts_ptr, lens_ptr, table_ptr, qs[0], qs[1], *strides,
                               os_[0], os_[1], table_stride, tokens, batch, heads, kv_heads, head_dim, pages, page_size,
                               max_pages, code, 1 if causal else 0, sm_scale)
    handle = _stream_of(device, stream)
    if workspace is None:
        need = lib().softmax_sequence_workspace_bytes(args)
        if need < 0:
            raise SoftmaxError(-need, what)
        workspace = _workspace_of(need, q, device, handle) if stream is None else \
            _new_tensor((need,), torch.uint8, q, stream)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{what}: workspace must be a contiguous tensor on {device}")
    st = call(args, workspace.data_ptr(), workspace.nbytes, handle)
    if st != OK:
        raise SoftmaxError(st, what)
    return out


def attention_varlen_fwd(q, k, v, q_starts, causal: bool = True, sm_scale: float | None = None, out=None, lse=None,
                         workspace=None, stream=None):
    """Attention forward over packed prompts of different lengths, with grouped
    heads: q [tokens, heads, head_dim], k and v [tokens, kv_heads, head_dim]
    (fp16 / bf16, head_dim 64 or 128, heads a multiple of kv_heads), sequence b
    in the rows q_starts[b] .. q_starts[b + 1] - 1 (an int32 CUDA tensor of
    batch + 1 offsets; no host synchronisation).  ``causal``: query i keeps keys
    0 .. i of its sequence, else all of them.  ``lse`` (optional, float32
    [tokens, heads]) receives the log of each row's sum of exponentials.  Rows of
    no sequence are not written (in a new ``out`` they are undefined).
    ``workspace`` (optional, a CUDA tensor of sequence_workspace_bytes) defaults to
    one that the thread keeps for the current stream (up to 64 MB each; a new one in
    a capture or with ``stream``); calls that share one must not run at the same time.
    Returns ``out``."""
    return _sequence_attention("attention_varlen_fwd", lib().softmax_attention_varlen_fwd, q, k, v, None, causal, sm_scale,
                               q_starts, out, lse, workspace, stream)


def attention_paged_fwd(q, k_cache, v_cache, page_table, kv_lens, q_starts, causal: bool = True,
                        sm_scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """Attention forward of new tokens (a chunk, drafts or single tokens) over
    a paged key/value cache that holds them already (see kv_cache_append): q
    [tokens, heads, head_dim] packed by q_starts as in attention_varlen_fwd,
    k_cache and v_cache [pages, page_size, kv_heads, head_dim] (any order of the
    strides; page_size a multiple of 8), page_table int32 [batch, max_pages],
    kv_lens int32 [batch], the keys of each sequence with its new ones.
    ``causal``: new token i of n keeps keys 0 .. kv_len - n + i, else all.  Other
    arguments as attention_varlen_fwd; returns ``out``."""
    return _sequence_attention("attention_paged_fwd", lib().softmax_attention_paged_fwd, q, k_cache, v_cache,
                               (page_table, kv_lens), causal, sm_scale, q_starts, out, lse, workspace, stream)


def sequence_workspace_bytes(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int, dtype,
                             page_size: int = 0, pages: int = 0, max_pages: int = 0, causal: bool = True) -> int:
    """Workspace bytes of attention_varlen_fwd (page_size 0) or attention_paged_fwd
    for these sizes on the current device."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else dtype
    args = SequenceArgs(tokens=tokens, batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, pages=pages,
                        page_size=page_size, max_pages=max_pages, dtype=code, causal=1 if causal else 0, sm_scale=1.0,
                        page_table=16 if page_size else None)
    n = lib().softmax_sequence_workspace_bytes(ctypes.byref(args))
    if n < 0:
        raise SoftmaxError(-n, "softmax_sequence_workspace_bytes")
    return n


def kv_cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q_starts, inv_freq=None, interleaved: bool = False,
                    q=None, q_out=None, stream=None):
    """Write the new tokens' keys and values [tokens, kv_heads, head_dim], packed
    by q_starts, to their places in the paged cache (kv_lens counts them
    already), and rotate on the way: with ``inv_freq`` (float32, rotary_dim / 2
    angles per position) the keys, and the queries ``q`` [tokens, heads,
    head_dim] if given, turn by their positions.  Pairs are (d, d + rotary_dim / 2),
    with ``interleaved`` (2d, 2d + 1).  Rotated queries go to ``q_out`` (default a
    new tensor; q itself rotates in place).  Returns q_out (None without q)."""
    import torch
    what = "kv_cache_append"
    k_ptr, (tokens, kv_heads, head_dim), ks, dtype, device, code = _first_operand(k, what, "k")
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return kv_cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q_starts, inv_freq, interleaved, q, q_out,
                                   stream)
    v_ptr, vsh, vs = _operand(v, what, "v", 3, dtype, device)
    kc_ptr, kcsh, kcs = _operand(k_cache, what, "k_cache", 4, dtype, device)
    vc_ptr, vcsh, vcs = _operand(v_cache, what, "v_cache", 4, dtype, device)
    if vsh != k.shape or kcsh != vcsh or kcsh[2] != kv_heads or kcsh[3] != head_dim:
        raise ValueError(f"{what}: k and v must be [tokens, kv_heads, head_dim] of the caches' last two sizes, the caches "
                         "of one shape")
    batch, max_pages, table_stride, starts_ptr, lens_ptr, table_ptr = _tables(what, page_table, kv_lens, q_starts, device)
    heads = q_ptr = out_ptr = 0
    qs = os_ = (0, 0)
    if q is not None:
        q_ptr, qsh, qs = _operand(q, what, "q", 3, dtype, device)
        if qsh[0] != tokens or qsh[2] != head_dim:
            raise ValueError(f"{what}: q must be [tokens, heads, head_dim] of k's tokens and head_dim")
        if q_out is None:
            q_out = _new_tensor(qsh, dtype, q, stream)
        out_ptr, osh, os_ = _operand(q_out, what, "q_out", 3, dtype, device)
        if osh != qsh:
            raise ValueError(f"{what}: q_out must have q's shape")
        heads = qsh[1]
    elif q_out is not None:
        raise ValueError(f"{what}: q_out without q")
    freq_ptr = rotary = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype is not torch.float32 or inv_freq.device != device:
            raise TypeError(f"{what}: inv_freq must be a float32 vector on {device}")
        freq_ptr, fsh, _ = _operand(inv_freq, what, "inv_freq", 1, torch.float32, device)
        rotary = 2 * fsh[0]
    args = _APPEND_PACK.pack(k_ptr, v_ptr, kc_ptr, vc_ptr, q_ptr, out_ptr, starts_ptr, lens_ptr, table_ptr, freq_ptr,
                             ks[0], ks[1], vs[0], vs[1], qs[0], qs[1], os_[0], os_[1], kcs[0], kcs[1], kcs[2], vcs[0],
                             vcs[1], vcs[2], table_stride, tokens, batch, heads, kv_heads, head_dim, kcsh[0], kcsh[1],
                             max_pages, rotary, 1 if interleaved else 0, code)
    st = lib().softmax_kv_cache_append(args, _stream_of(device, stream))
    if st != OK:
        raise SoftmaxError(st, what)
    return q_out


def host_workspace_bytes(rows: int, cols: int, row_stride: int, dtype, chunk_bytes: int = 0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else dtype
    n = lib().softmax_host_workspace_bytes(rows, cols, row_stride, code, chunk_bytes)
    if n < 0:
        raise SoftmaxError(-n, "softmax_host_workspace_bytes")
    return n


def softmax_fwd_host(x, out=None, workspace=None, stream=None, zero_copy: bool = False):
    """Row softmax of a 2-D CPU tensor (pinned for overlapping copies),
    written to ``out`` (a CPU tensor, default a new pinned one) through the
    library's chunked copy / softmax / copy pipeline on the current CUDA
    device.  ``workspace`` (a CUDA tensor) defaults to a new one of
    softmax_host_workspace_bytes.  ``zero_copy=True`` passes no workspace:
    the kernels read and write the host buffers in place (they must be memory
    the device reaches directly).  Synchronises ``stream`` before returning."""
    import torch
    if not isinstance(x, torch.Tensor) or x.is_cuda or x.dim() != 2:
        raise TypeError("softmax_fwd_host needs a 2-D CPU tensor")
    rows, cols = x.shape
    if cols > 1 and x.stride(1) != 1:
        raise ValueError("the last dimension must be contiguous (stride 1)")
    row_stride = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    code = _torch_dtype_code(x)
    if out is None:
        out = torch.empty_strided((rows, cols), (row_stride, 1), dtype=x.dtype, pin_memory=True)
    elif out.shape != x.shape or out.dtype != x.dtype or out.is_cuda or (rows > 1 and out.stride(0) != row_stride):
        raise ValueError("out must be a CPU tensor with x's shape, dtype and row stride")
    if zero_copy:
        ws_ptr, ws_bytes = None, 0
    else:
        if workspace is None:
            workspace = torch.empty(max(host_workspace_bytes(rows, cols, row_stride, code), 1), dtype=torch.uint8,
                                    device="cuda")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    s = stream if stream is not None else torch.cuda.current_stream()
    handle = s.cuda_stream if hasattr(s, "cuda_stream") else int(s)
    st = lib().softmax_fwd_host(x.data_ptr(), out.data_ptr(), rows, cols, row_stride, code, ws_ptr, ws_bytes,
                                handle)
    if st != OK:
        raise SoftmaxError(st, "softmax_fwd_host")
    torch.cuda.current_stream().synchronize() if stream is None else s.synchronize()
    return out


def autotune(x, out=None, stream=None, iters: int = 20) -> dict:
    """softmax_autotune on a tensor (``out`` must be another buffer): time the
    candidate launch shapes and cache the fastest for calls of this shape."""
    import torch
    rows, cols, row_stride, code, out = _prepare(x, out, "autotune")
    if out.data_ptr() == x.data_ptr():
        raise ValueError("autotune needs an out buffer other than x")
    with torch.cuda.device(x.device):
        return autotune_ptr(x.data_ptr(), out.data_ptr(), rows, cols, row_stride, code, _stream_handle(x, stream),
                            iters)


def plan(in_addr: int, out_addr: int, rows: int, cols: int, row_stride: int, dtype,
         num_sms: int = 0) -> dict:
    """The launch softmax_fwd would make (host only when num_sms > 0)."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else dtype
    p = Plan()
    st = lib().softmax_plan(in_addr, out_addr, rows, cols, row_stride, code, num_sms, ctypes.byref(p))
    if st != OK:
        raise SoftmaxError(st, "softmax_plan")
    return p.as_dict()


def set_force_path(path: int, threads: int = 0, vpt: int = 0, group: int = 0) -> None:
    st = lib().softmax_set_force_path(path, threads, vpt, group)
    if st != OK:
        raise SoftmaxError(st, "softmax_set_force_path")


def last_path() -> int:
    return lib().softmax_last_path()


def check_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    handle = s.cuda_stream if hasattr(s, "cuda_stream") else int(s)
    return lib().softmax_check_device_error(handle)


def set_wait_test(wait_limit_ns: int = 0, starve: bool = False) -> None:
    lib().softmax_set_wait_test(wait_limit_ns, 1 if starve else 0)


def attention_plan(batch: int, heads: int, n_ctx: int, head_dim: int = 128, dtype="f16", causal: bool = True,
                   num_sms: int = 0) -> dict:
    """The launch softmax_attention_fwd makes for a shape (host only when
    num_sms > 0); raises SoftmaxError for arguments the call would refuse."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else dtype
    p = AttentionPlan()
    st = lib().softmax_attention_plan(batch, heads, n_ctx, head_dim, code, 1 if causal else 0, num_sms,
                                      ctypes.byref(p))
    if st != OK:
        raise SoftmaxError(st, "softmax_attention_plan")
    return p.as_dict()


def set_attention_wait_test(starve: bool = False) -> None:
    """Test hook of the attention calls: leave the first Q barrier (or key tile's) of
    every block unarmed so that its bounded wait runs out (see set_wait_test for the limit)."""
    lib().softmax_attention_set_wait_test(1 if starve else 0)


def set_launch_overlap(enable: bool = True) -> None:
    """Programmatic dependent launch on (default) or off, process-wide."""
    lib().softmax_set_launch_overlap(1 if enable else 0)


def autotune_ptr(in_ptr: int, out_ptr: int, rows: int, cols: int, row_stride: int, dtype: int, stream: int = 0,
                 iters: int = 20) -> dict:
    """Time the candidate launch shapes for this call and cache the fastest
    (raises on a bad status).  Returns the kept plan and the timings."""
    r = TuneResult()
    st = lib().softmax_autotune(in_ptr, out_ptr, rows, cols, row_stride, dtype, stream, iters, ctypes.byref(r))
    if st != OK:
        raise SoftmaxError(st, "softmax_autotune")
    return {"plan": r.plan.as_dict(), "best_us": r.best_us, "auto_us": r.auto_us, "candidates": r.candidates}


def tune_candidates(in_addr: int, out_addr: int, rows: int, cols: int, row_stride: int, dtype) -> list:
    """The (path, threads, vpt, group) shapes softmax_autotune would time."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else dtype
    n = lib().softmax_tune_candidates(in_addr, out_addr, rows, cols, row_stride, code, 0, None, 0)
    if n < 0:
        raise SoftmaxError(-n, "softmax_tune_candidates")
    arr = (Shape * max(n, 1))()
    lib().softmax_tune_candidates(in_addr, out_addr, rows, cols, row_stride, code, 0, arr, n)
    return [arr[i].as_tuple() for i in range(n)]


def autotune_size() -> int:
    return lib().softmax_autotune_size()


def autotune_clear() -> None:
    lib().softmax_autotune_clear()


def abi_version() -> int:
    return lib().softmax_abi_version()
