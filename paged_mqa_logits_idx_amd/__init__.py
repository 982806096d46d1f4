"""Python binding of the paged MQA-logits indexer library (libidx_paged_mqa.so).

Argument marshalling only: every step of the computation runs in the library's
HIP kernels.  The functions carry the C-ABI names and argument order; they
accept torch device tensors (or raw device addresses as ints) and pass their
addresses and sizes through ctypes.  torch supplies device memory and streams.

The library must be built in-tree first (``python paged_mqa_logits_idx_amd/_build.py``
or ``__graft_entry__.build()``); importing this module without it raises.
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path

import torch  # loads the HIP runtime the library binds to (same soname)

LIB_PATH = Path(__file__).resolve().parent / "libidx_paged_mqa.so"

NUM_HEADS = 64
HEAD_DIM = 128
PAGE_POSITIONS = 64
FP8_PAGE_KEY_BYTES = PAGE_POSITIONS * HEAD_DIM          # 8192
FP8_PAGE_SCALE_BYTES = PAGE_POSITIONS * 4               # 256
FP8_FUSED_PAGE_BYTES = FP8_PAGE_KEY_BYTES + FP8_PAGE_SCALE_BYTES  # 8448
BF16_PAGE_BYTES = PAGE_POSITIONS * HEAD_DIM * 2         # 16384
LATENT_DIM = 512

IDX_NORM_OFF = 1
IDX_ROPE_LEADING = 2
IDX_ROPE_HALVES = 4

IDX_OK = 0
IDX_ERR_NULL = -1
IDX_ERR_UNSUPPORTED = -2
IDX_ERR_SHAPE = -3
IDX_ERR_ALIGN = -4
IDX_ERR_LAUNCH = -5

_SYMBOLS = (
    "idx_paged_mqa_logits_fp8",
    "idx_paged_mqa_logits_bf16",
    "idx_paged_mqa_logits_varlen_fp8",
    "idx_paged_mqa_logits_varlen_bf16",
    "idx_topk_logits",
    "idx_paged_mqa_topk_fp8",
    "idx_paged_mqa_topk_bf16",
    "idx_store_keys_fp8",
    "idx_store_keys_bf16",
    "idx_norm_rope",
    "idx_norm_rope_store_fp8",
    "idx_norm_rope_store_bf16",
    "idx_load_slots_fp8",
    "idx_load_slots_bf16",
    "idx_latent_attention_fp8",
    "idx_latent_attention_bf16",
    "idx_latent_attention_workspace",
    "idx_status_string",
    "idx_abi_version",
)


class IdxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


def _load() -> ctypes.CDLL:
    if not LIB_PATH.exists():
        raise ImportError(
            f"{LIB_PATH} is missing: build the HIP library first "
            "(python paged_mqa_logits_idx_amd/_build.py)")
    lib = ctypes.CDLL(str(LIB_PATH))
    argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_void_p,
    ]
    for name in ("idx_paged_mqa_logits_fp8", "idx_paged_mqa_logits_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    for name in ("idx_paged_mqa_logits_varlen_fp8", "idx_paged_mqa_logits_varlen_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = argtypes[:4] + [ctypes.c_void_p, ctypes.c_int32] + argtypes[4:]
        fn.restype = ctypes.c_int
    lib.idx_topk_logits.argtypes = [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.idx_topk_logits.restype = ctypes.c_int
    for name in ("idx_paged_mqa_topk_fp8", "idx_paged_mqa_topk_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = argtypes[:-1] + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p]
        fn.restype = ctypes.c_int
    lib.idx_store_keys_fp8.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
    lib.idx_store_keys_fp8.restype = ctypes.c_int
    lib.idx_store_keys_bf16.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_void_p]
    lib.idx_store_keys_bf16.restype = ctypes.c_int
    ptr, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    rotation = [i32, i32, ctypes.c_uint32, ctypes.c_float, i64]  # head_dim, rope_dim, flags, eps, row stride
    for name, types in (
            ("idx_norm_rope", [ptr] * 5 + [i64, i32] + rotation + [ptr]),
            ("idx_norm_rope_store_fp8", [ptr] * 5 + [i64] + rotation + [ptr, ptr, i64, i64, i64, ptr]),
            ("idx_norm_rope_store_bf16", [ptr] * 5 + [i64] + rotation + [ptr, i64, i64, ptr]),
            ("idx_load_slots_fp8", [ptr] * 3 + [i64, i32, i64, i64, i64, ptr, i64, ptr]),
            ("idx_load_slots_bf16", [ptr] * 2 + [i64, i32, i64, i64, ptr, i64, ptr]),
            ("idx_latent_attention_fp8", [ptr] * 5 + [i32] + [ptr] * 5 + [i32] * 4 + [i64] * 4
             + [i32, ctypes.c_float, ptr, i64, ptr]),
            ("idx_latent_attention_bf16", [ptr] * 4 + [i32] + [ptr] * 5 + [i32] * 4 + [i64] * 3
             + [i32, ctypes.c_float, ptr, i64, ptr])):
        fn = getattr(lib, name)
        fn.argtypes = types
        fn.restype = ctypes.c_int
    lib.idx_latent_attention_workspace.argtypes = [i32] * 4
    lib.idx_latent_attention_workspace.restype = i64
    lib.idx_status_string.argtypes = [ctypes.c_int]
    lib.idx_status_string.restype = ctypes.c_char_p
    lib.idx_abi_version.argtypes = []
    lib.idx_abi_version.restype = ctypes.c_int
    return lib


_lib = _load()


def idx_status_string(status: int) -> str:
    return _lib.idx_status_string(int(status)).decode()


def idx_abi_version() -> int:
    return int(_lib.idx_abi_version())


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if x.device.type != "cuda":
            raise ValueError("tensors passed to the indexer library must be device tensors")
        return x.data_ptr()
    return int(x)


def _check(name: str, x, dtype, dense_rows: bool = False) -> None:
    """A tensor argument must have the element type the kernels read and the
    dense layout they assume: contiguous, or (``dense_rows``: tables and logits,
    whose row stride is passed separately) unit stride along its last dim.
    Raw addresses are passed through unchecked."""
    if not isinstance(x, torch.Tensor):
        return
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    ok = (x.dim() == 0 or x.stride(-1) == 1 or x.shape[-1] <= 1) if dense_rows else x.is_contiguous()
    if not ok:
        raise ValueError(f"{name} must be " + ("unit-stride along its last dim" if dense_rows
                                                 else "contiguous"))


def _check_logits_args(q, kv_pages, kscale, page_table, seqlens, weights, out):
    _check("q", q, torch.bfloat16)
    if isinstance(kv_pages, torch.Tensor) and not kv_pages.is_contiguous():
        raise ValueError("kv_pages must be contiguous")
    if isinstance(kscale, torch.Tensor):
        _check("kscale", kscale, torch.float32)
    _check("page_table", page_table, torch.int32, dense_rows=True)
    _check("seqlens", seqlens, torch.int32)
    _check("weights", weights, torch.float32)
    _check("out", out, torch.float32)


def _stream_handle(stream, device) -> int | None:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _call(name, q, kv_pages, kscale, page_table, seqlens, weights, out, *, rows, num_heads,
          head_dim, table_width, num_pages, kv_page_stride, kscale_page_stride,
          page_table_row_stride, stream, check):
    _check_logits_args(q, kv_pages, kscale, page_table, seqlens, weights, out)
    dev = q.device if isinstance(q, torch.Tensor) else None
    fn = getattr(_lib, name)
    status = fn(_addr(q), _addr(kv_pages), _addr(kscale), _addr(page_table), _addr(seqlens),
                _addr(weights), _addr(out), int(rows), int(num_heads), int(head_dim),
                int(table_width), int(num_pages), int(kv_page_stride), int(kscale_page_stride),
                int(page_table_row_stride), _stream_handle(stream, dev))
    if check and status != IDX_OK:
        raise IdxError(status, f"{name}: {idx_status_string(status)}")
    return status


def _dims(q, page_table, table_width, rows, num_heads, head_dim, page_table_row_stride):
    if isinstance(q, torch.Tensor):
        if rows is None:
            rows = q.shape[0]
        if num_heads is None:
            num_heads = q.shape[1] if q.dim() == 3 else NUM_HEADS
        if head_dim is None:
            head_dim = q.shape[2] if q.dim() == 3 else HEAD_DIM
    if table_width is None:
        if not (isinstance(page_table, torch.Tensor) and page_table.dim() == 2):
            raise ValueError("table_width is required unless page_table is a 2-D tensor")
        table_width = page_table.shape[1]
    if page_table_row_stride is None:
        if not (isinstance(page_table, torch.Tensor) and page_table.dim() == 2):
            raise ValueError("page_table_row_stride is required unless page_table is a 2-D tensor")
        page_table_row_stride = 0 if page_table.shape[0] == 1 and rows != 1 else page_table.stride(0)
    return rows, num_heads, head_dim, table_width, page_table_row_stride


def idx_paged_mqa_logits_fp8(q, kv_pages, kscale, page_table, seqlens, weights, out, *,
                             num_pages, kv_page_stride=FP8_FUSED_PAGE_BYTES,
                             kscale_page_stride=FP8_FUSED_PAGE_BYTES, table_width=None,
                             page_table_row_stride=None, rows=None, num_heads=None,
                             head_dim=None, stream=None, check=True) -> int:
    """out[b, p] = sum_h w[b,h] * ReLU(s_p * <q[b,h], k_p>) for p < seqlens[b], else -inf.

    fp8 (e4m3fn) keys with a per-position fp32 scale.  ``kscale`` is a tensor or
    a device address; for the fused 8448-byte block pass
    ``kv_pages.data_ptr() + 8192``.  Returns the library status (raises
    IdxError on failure when ``check``).
    """
    rows, num_heads, head_dim, table_width, pts = _dims(
        q, page_table, table_width, rows, num_heads, head_dim, page_table_row_stride)
    return _call("idx_paged_mqa_logits_fp8", q, kv_pages, kscale, page_table, seqlens, weights,
                 out, rows=rows, num_heads=num_heads, head_dim=head_dim, table_width=table_width,
                 num_pages=num_pages, kv_page_stride=kv_page_stride,
                 kscale_page_stride=kscale_page_stride, page_table_row_stride=pts, stream=stream,
                 check=check)


def idx_paged_mqa_logits_bf16(q, kv_pages, kscale, page_table, seqlens, weights, out, *,
                              num_pages, kv_page_stride=BF16_PAGE_BYTES, kscale_page_stride=0,
                              table_width=None, page_table_row_stride=None, rows=None,
                              num_heads=None, head_dim=None, stream=None, check=True) -> int:
    """Same as :func:`idx_paged_mqa_logits_fp8` with bf16 keys and s_p = 1 (kscale must be None)."""
    rows, num_heads, head_dim, table_width, pts = _dims(
        q, page_table, table_width, rows, num_heads, head_dim, page_table_row_stride)
    return _call("idx_paged_mqa_logits_bf16", q, kv_pages, kscale, page_table, seqlens, weights,
                 out, rows=rows, num_heads=num_heads, head_dim=head_dim, table_width=table_width,
                 num_pages=num_pages, kv_page_stride=kv_page_stride,
                 kscale_page_stride=kscale_page_stride, page_table_row_stride=pts, stream=stream,
                 check=check)


def _call_varlen(name, q, kv_pages, kscale, page_table, row_table, seqlens, weights, out, *,
                 num_tables, num_pages, table_width, page_table_row_stride, kv_page_stride,
                 kscale_page_stride, rows, num_heads, head_dim, stream, check):
    if isinstance(q, torch.Tensor):
        rows = q.shape[0] if rows is None else rows
    num_heads = NUM_HEADS if num_heads is None else num_heads
    head_dim = HEAD_DIM if head_dim is None else head_dim
    _check_logits_args(q, kv_pages, kscale, page_table, seqlens, weights, out)
    _check("row_table", row_table, torch.int32)
    dev = q.device if isinstance(q, torch.Tensor) else None
    status = getattr(_lib, name)(
        _addr(q), _addr(kv_pages), _addr(kscale), _addr(page_table), _addr(row_table),
        int(num_tables), _addr(seqlens), _addr(weights), _addr(out), int(rows), int(num_heads),
        int(head_dim), int(table_width), int(num_pages), int(kv_page_stride),
        int(kscale_page_stride), int(page_table_row_stride), _stream_handle(stream, dev))
    if check and status != IDX_OK:
        raise IdxError(status, f"{name}: {idx_status_string(status)}")
    return status


def idx_paged_mqa_logits_varlen_fp8(q, kv_pages, kscale, page_table, row_table, seqlens, weights,
                                    out, *, num_tables, num_pages, table_width,
                                    page_table_row_stride=None,
                                    kv_page_stride=FP8_FUSED_PAGE_BYTES,
                                    kscale_page_stride=FP8_FUSED_PAGE_BYTES, rows=None,
                                    num_heads=None, head_dim=None, stream=None,
                                    check=True) -> int:
    """Several requests' query rows in one call: row b uses table row_table[b]
    (at page_table + row_table[b]*page_table_row_stride) and its own seqlen."""
    pts = table_width if page_table_row_stride is None else page_table_row_stride
    return _call_varlen("idx_paged_mqa_logits_varlen_fp8", q, kv_pages, kscale, page_table,
                        row_table, seqlens, weights, out, num_tables=num_tables,
                        num_pages=num_pages, table_width=table_width, page_table_row_stride=pts,
                        kv_page_stride=kv_page_stride, kscale_page_stride=kscale_page_stride,
                        rows=rows, num_heads=num_heads, head_dim=head_dim, stream=stream,
                        check=check)


def idx_paged_mqa_logits_varlen_bf16(q, kv_pages, kscale, page_table, row_table, seqlens, weights,
                                     out, *, num_tables, num_pages, table_width,
                                     page_table_row_stride=None, kv_page_stride=BF16_PAGE_BYTES,
                                     kscale_page_stride=0, rows=None, num_heads=None,
                                     head_dim=None, stream=None, check=True) -> int:
    """bf16-key counterpart of :func:`idx_paged_mqa_logits_varlen_fp8`."""
    pts = table_width if page_table_row_stride is None else page_table_row_stride
    return _call_varlen("idx_paged_mqa_logits_varlen_bf16", q, kv_pages, kscale, page_table,
                        row_table, seqlens, weights, out, num_tables=num_tables,
                        num_pages=num_pages, table_width=table_width, page_table_row_stride=pts,
                        kv_page_stride=kv_page_stride, kscale_page_stride=kscale_page_stride,
                        rows=rows, num_heads=num_heads, head_dim=head_dim, stream=stream,
                        check=check)


def idx_topk_logits(logits, seqlens, topk_idx, topk_val=None, *, k=None, rows=None, ncols=None,
                    row_stride=None, stream=None, check=True) -> int:
    """Per row b, the k largest of logits[b, :clamp(seqlens[b], 0, ncols)] (equal
    values by lower position, NaN last), in ascending position order, -1 padded.

    ``topk_idx`` int32 [rows, k]; ``topk_val`` optional fp32 [rows, k].  Dims
    default to the tensors' shapes.
    """
    if isinstance(logits, torch.Tensor):
        rows = logits.shape[0] if rows is None else rows
        ncols = logits.shape[1] if ncols is None else ncols
        row_stride = logits.stride(0) if row_stride is None else row_stride
    if k is None:
        k = topk_idx.shape[1]
    _check("logits", logits, torch.float32, dense_rows=True)
    _check("seqlens", seqlens, torch.int32)
    _check("topk_idx", topk_idx, torch.int32)
    _check("topk_val", topk_val, torch.float32)
    dev = topk_idx.device if isinstance(topk_idx, torch.Tensor) else None
    status = _lib.idx_topk_logits(_addr(logits), int(row_stride), _addr(seqlens), int(rows),
                                  int(ncols), int(k), _addr(topk_idx), _addr(topk_val),
                                  _stream_handle(stream, dev))
    if check and status != IDX_OK:
        raise IdxError(status, f"idx_topk_logits: {idx_status_string(status)}")
    return status


def _call_topk(name, q, kv_pages, kscale, page_table, seqlens, weights, logits, topk_idx, topk_val,
               *, k, rows, num_heads, head_dim, table_width, num_pages, kv_page_stride,
               kscale_page_stride, page_table_row_stride, stream, check):
    rows, num_heads, head_dim, table_width, pts = _dims(
        q, page_table, table_width, rows, num_heads, head_dim, page_table_row_stride)
    if k is None:
        k = topk_idx.shape[1]
    _check_logits_args(q, kv_pages, kscale, page_table, seqlens, weights, logits)
    _check("topk_idx", topk_idx, torch.int32)
    _check("topk_val", topk_val, torch.float32)
    dev = q.device if isinstance(q, torch.Tensor) else None
    status = getattr(_lib, name)(
        _addr(q), _addr(kv_pages), _addr(kscale), _addr(page_table), _addr(seqlens),
        _addr(weights), _addr(logits), int(rows), int(num_heads), int(head_dim), int(table_width),
        int(num_pages), int(kv_page_stride), int(kscale_page_stride), int(pts), int(k),
        _addr(topk_idx), _addr(topk_val), _stream_handle(stream, dev))
    if check and status != IDX_OK:
        raise IdxError(status, f"{name}: {idx_status_string(status)}")
    return status


def idx_paged_mqa_topk_fp8(q, kv_pages, kscale, page_table, seqlens, weights, logits, topk_idx,
                           topk_val=None, *, num_pages, k=None,
                           kv_page_stride=FP8_FUSED_PAGE_BYTES,
                           kscale_page_stride=FP8_FUSED_PAGE_BYTES, table_width=None,
                           page_table_row_stride=None, rows=None, num_heads=None, head_dim=None,
                           stream=None, check=True) -> int:
    """Logits into ``logits`` (only positions p < seqlens[b] defined afterwards),
    then their top-k into ``topk_idx`` / ``topk_val``, in one call."""
    return _call_topk("idx_paged_mqa_topk_fp8", q, kv_pages, kscale, page_table, seqlens, weights,
                      logits, topk_idx, topk_val, k=k, rows=rows, num_heads=num_heads,
                      head_dim=head_dim, table_width=table_width, num_pages=num_pages,
                      kv_page_stride=kv_page_stride, kscale_page_stride=kscale_page_stride,
                      page_table_row_stride=page_table_row_stride, stream=stream, check=check)


def idx_paged_mqa_topk_bf16(q, kv_pages, kscale, page_table, seqlens, weights, logits, topk_idx,
                            topk_val=None, *, num_pages, k=None, kv_page_stride=BF16_PAGE_BYTES,
                            kscale_page_stride=0, table_width=None, page_table_row_stride=None,
                            rows=None, num_heads=None, head_dim=None, stream=None,
                            check=True) -> int:
    """bf16-key counterpart of :func:`idx_paged_mqa_topk_fp8` (kscale must be None)."""
    return _call_topk("idx_paged_mqa_topk_bf16", q, kv_pages, kscale, page_table, seqlens, weights,
                      logits, topk_idx, topk_val, k=k, rows=rows, num_heads=num_heads,
                      head_dim=head_dim, table_width=table_width, num_pages=num_pages,
                      kv_page_stride=kv_page_stride, kscale_page_stride=kscale_page_stride,
                      page_table_row_stride=page_table_row_stride, stream=stream, check=check)


def idx_store_keys_fp8(keys, slots, kv_pages, kscale, *, num_pages, n=None,
                       kv_page_stride=FP8_FUSED_PAGE_BYTES, kscale_page_stride=FP8_FUSED_PAGE_BYTES,
                       stream=None, check=True) -> int:
    """Quantise bf16 keys [n, 128] (scale = amax/448, e4m3fn codes) into pool slots.

    ``slots`` is int64 [n] (64*page + position; out of range skips the key).
    ``kscale`` is a tensor or a device address (fused block: kv_pages + 8192).
    """
    if n is None:
        n = keys.shape[0]
    _check("keys", keys, torch.bfloat16)
    _check("slots", slots, torch.int64)
    if isinstance(kscale, torch.Tensor):
        _check("kscale", kscale, torch.float32)
    if isinstance(kv_pages, torch.Tensor) and not kv_pages.is_contiguous():
        raise ValueError("kv_pages must be contiguous")
    dev = keys.device if isinstance(keys, torch.Tensor) else None
    status = _lib.idx_store_keys_fp8(_addr(keys), _addr(slots), int(n), _addr(kv_pages),
                                     _addr(kscale), int(num_pages), int(kv_page_stride),
                                     int(kscale_page_stride), _stream_handle(stream, dev))
    if check and status != IDX_OK:
        raise IdxError(status, f"idx_store_keys_fp8: {idx_status_string(status)}")
    return status


def idx_store_keys_bf16(keys, slots, kv_pages, *, num_pages, n=None, kv_page_stride=BF16_PAGE_BYTES,
                        stream=None, check=True) -> int:
    """Copy bf16 keys [n, 128] into 16384-byte bf16 pages at the given slots."""
    if n is None:
        n = keys.shape[0]
    _check("keys", keys, torch.bfloat16)
    _check("slots", slots, torch.int64)
    if isinstance(kv_pages, torch.Tensor) and not kv_pages.is_contiguous():
        raise ValueError("kv_pages must be contiguous")
    dev = keys.device if isinstance(keys, torch.Tensor) else None
    status = _lib.idx_store_keys_bf16(_addr(keys), _addr(slots), int(n), _addr(kv_pages),
                                      int(num_pages), int(kv_page_stride), _stream_handle(stream, dev))
    if check and status != IDX_OK:
        raise IdxError(status, f"idx_store_keys_bf16: {idx_status_string(status)}")
    return status


def _device_of(named) -> torch.device | None:
    """The one device of a call's tensors ((name, tensor or address) pairs)."""
    dev = None
    for name, x in named:
        if isinstance(x, torch.Tensor):
            if x.device.type != "cuda":
                raise ValueError("tensors passed to the indexer library must be device tensors")
            if dev is None:
                dev = x.device
            elif x.device != dev:
                raise ValueError(f"{name} is on {x.device}, the arguments before it on {dev}")
    return dev


def _launch(name, dev, stream, check, *args) -> int:
    """Calls the library with ``args`` and the stream, on the tensors' device
    (whatever the current one is)."""
    fn, handle = getattr(_lib, name), _stream_handle(stream, dev)
    if dev is None or dev.index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if check and status != IDX_OK:
        raise IdxError(status, f"{name}: {idx_status_string(status)}")
    return status


def _check_rows(name, x, dim, width=None) -> None:
    """A bf16 tensor of ``dim`` dims whose rows (all dims but the first) are
    dense; the first dim's stride is free."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {x.dtype}")
    if x.dim() != dim or (width is not None and x.shape[-1] != width):
        raise ValueError(f"{name} must have {dim} dims" + ("" if width is None else f", the last of {width}")
                         + f", got {tuple(x.shape)}")
    dense = 1
    for size, stride in zip(reversed(x.shape[1:]), reversed(x.stride()[1:])):
        if size > 1 and stride != dense:
            raise ValueError(f"{name} must be dense behind its first dim")
        dense *= size


def _row_stride(x) -> int:
    """Elements between the rows of a tensor checked by ``_check_rows``."""
    return x.stride(0) if x.shape[0] > 1 else math.prod(x.shape[1:])


def _rotation(x, positions, inv_freq, weight, norm, leading, halves):
    """Checks the norm and rotation's arguments; (head_dim, rope_dim, flags)."""
    n, head_dim = x.shape[0], x.shape[-1]
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    _check("positions", positions, torch.int64)
    _check("inv_freq", inv_freq, torch.float32)
    _check("weight", weight, torch.float32)
    if positions is not None and positions.shape != (n,):
        raise ValueError(f"positions must be [{n}], got {list(positions.shape)}")
    if inv_freq is not None and inv_freq.dim() != 1:
        raise ValueError("inv_freq must have one dim")
    if weight is not None and weight.shape != (head_dim,):
        raise ValueError(f"weight must be [{head_dim}], got {list(weight.shape)}")
    if weight is not None and not norm:
        raise ValueError("weight goes with the norm")
    flags = (0 if norm else IDX_NORM_OFF) | (IDX_ROPE_LEADING if leading else 0) | (IDX_ROPE_HALVES if halves else 0)
    return head_dim, 0 if inv_freq is None else 2 * inv_freq.shape[0], flags


def _check_pool(kv_pages, kscale, num_pages, page_bytes, kv_page_stride, kscale_page_stride) -> None:
    """A pool given as tensors must hold the pages (``page_bytes`` of values
    each) that it is said to hold."""
    if isinstance(kv_pages, torch.Tensor):
        if not kv_pages.is_contiguous():
            raise ValueError("kv_pages must be contiguous")
        if num_pages > 0 and kv_pages.numel() * kv_pages.element_size() < (num_pages - 1) * kv_page_stride + page_bytes:
            raise ValueError(f"kv_pages is shorter than {num_pages} pages of {kv_page_stride} bytes")
    if isinstance(kscale, torch.Tensor):
        _check("kscale", kscale, torch.float32)
        if num_pages > 0 and kscale.numel() * 4 < (num_pages - 1) * kscale_page_stride + 4 * PAGE_POSITIONS:
            raise ValueError(f"kscale is shorter than {num_pages} pages of {kscale_page_stride} bytes")


def _check_slots(slots, n) -> None:
    _check("slots", slots, torch.int64)
    if isinstance(slots, torch.Tensor) and slots.shape != (n,):
        raise ValueError(f"slots must be [{n}], got {list(slots.shape)}")


def idx_norm_rope(x, positions, inv_freq, out, *, weight=None, eps=1e-6, norm=True, leading=False,
                  halves=False, stream=None, check=True) -> int:
    """RMS norm (times ``weight``) and rotation of the vectors of bf16 ``x``
    [n, heads, D] (D 64, 128, 256 or 512; the first dim may be strided), head by
    head, into bf16 ``out`` (contiguous; may be ``x``).

    Token t's rotated values (the last 2*len(inv_freq) of D, or the first with
    ``leading``; neighbours, or halves with ``halves``) turn by positions[t] *
    inv_freq[j].  ``positions`` int64 [n] and ``inv_freq`` fp32; both None: no
    rotation.  ``norm=False``: only the rotation.
    """
    _check_rows("x", x, 3)
    _check("out", out, torch.bfloat16)
    if out.shape != x.shape:
        raise ValueError(f"out must be {list(x.shape)}, got {list(out.shape)}")
    head_dim, rope_dim, flags = _rotation(x, positions, inv_freq, weight, norm, leading, halves)
    dev = _device_of((("x", x), ("positions", positions), ("inv_freq", inv_freq), ("weight", weight), ("out", out)))
    return _launch("idx_norm_rope", dev, stream, check, _addr(x), _addr(weight), _addr(positions), _addr(inv_freq),
                   _addr(out), x.shape[0], x.shape[1], head_dim, rope_dim, flags, eps, _row_stride(x))


def idx_norm_rope_store_fp8(x, positions, inv_freq, slots, kv_pages, kscale, *, num_pages, weight=None,
                            eps=1e-6, norm=True, leading=False, halves=False, kv_page_stride=None,
                            kscale_page_stride=None, stream=None, check=True) -> int:
    """Norm and rotation (as :func:`idx_norm_rope`) of bf16 vectors [n, D] (D 128:
    index keys, 512: latents), quantised (scale = amax/448, e4m3fn codes) into
    pool slots in the same pass.

    ``slots`` int64 [n] (64*page + position; out of range skips the token).  The
    strides default to the fused block of 64*D + 256 bytes; ``kscale`` is a
    tensor or a device address (fused block: kv_pages + 64*D).
    """
    _check_rows("x", x, 2)
    head_dim, rope_dim, flags = _rotation(x, positions, inv_freq, weight, norm, leading, halves)
    fused = PAGE_POSITIONS * (head_dim + 4)
    kv_page_stride = fused if kv_page_stride is None else kv_page_stride
    kscale_page_stride = fused if kscale_page_stride is None else kscale_page_stride
    _check_slots(slots, x.shape[0])
    _check_pool(kv_pages, kscale, num_pages, PAGE_POSITIONS * head_dim, kv_page_stride, kscale_page_stride)
    dev = _device_of((("x", x), ("positions", positions), ("inv_freq", inv_freq), ("weight", weight),
                      ("slots", slots), ("kv_pages", kv_pages), ("kscale", kscale)))
    return _launch("idx_norm_rope_store_fp8", dev, stream, check, _addr(x), _addr(weight), _addr(positions),
                   _addr(inv_freq), _addr(slots), x.shape[0], head_dim, rope_dim, flags, eps, _row_stride(x),
                   _addr(kv_pages), _addr(kscale), num_pages, kv_page_stride, kscale_page_stride)


def idx_norm_rope_store_bf16(x, positions, inv_freq, slots, kv_pages, *, num_pages, weight=None, eps=1e-6,
                             norm=True, leading=False, halves=False, kv_page_stride=None, stream=None,
                             check=True) -> int:
    """bf16 counterpart of :func:`idx_norm_rope_store_fp8`: pages of 128*D bytes."""
    _check_rows("x", x, 2)
    head_dim, rope_dim, flags = _rotation(x, positions, inv_freq, weight, norm, leading, halves)
    kv_page_stride = 2 * PAGE_POSITIONS * head_dim if kv_page_stride is None else kv_page_stride
    _check_slots(slots, x.shape[0])
    _check_pool(kv_pages, None, num_pages, 2 * PAGE_POSITIONS * head_dim, kv_page_stride, 0)
    dev = _device_of((("x", x), ("positions", positions), ("inv_freq", inv_freq), ("weight", weight),
                      ("slots", slots), ("kv_pages", kv_pages)))
    return _launch("idx_norm_rope_store_bf16", dev, stream, check, _addr(x), _addr(weight), _addr(positions),
                   _addr(inv_freq), _addr(slots), x.shape[0], head_dim, rope_dim, flags, eps, _row_stride(x),
                   _addr(kv_pages), num_pages, kv_page_stride)


def idx_load_slots_fp8(kv_pages, kscale, slots, out, *, num_pages, kv_page_stride=None,
                       kscale_page_stride=None, stream=None, check=True) -> int:
    """out[t] = bf16(code * scale) of pool slot slots[t], for bf16 ``out`` [n, D]
    (D 128 or 512; rows may be strided).  A slot out of range leaves its row."""
    _check_rows("out", out, 2)
    head_dim = out.shape[1]
    fused = PAGE_POSITIONS * (head_dim + 4)
    kv_page_stride = fused if kv_page_stride is None else kv_page_stride
    kscale_page_stride = fused if kscale_page_stride is None else kscale_page_stride
    _check_slots(slots, out.shape[0])
    _check_pool(kv_pages, kscale, num_pages, PAGE_POSITIONS * head_dim, kv_page_stride, kscale_page_stride)
    dev = _device_of((("out", out), ("slots", slots), ("kv_pages", kv_pages), ("kscale", kscale)))
    return _launch("idx_load_slots_fp8", dev, stream, check, _addr(kv_pages), _addr(kscale), _addr(slots),
                   out.shape[0], head_dim, num_pages, kv_page_stride, kscale_page_stride, _addr(out), _row_stride(out))


def idx_load_slots_bf16(kv_pages, slots, out, *, num_pages, kv_page_stride=None, stream=None, check=True) -> int:
    """bf16 counterpart of :func:`idx_load_slots_fp8`."""
    _check_rows("out", out, 2)
    head_dim = out.shape[1]
    kv_page_stride = 2 * PAGE_POSITIONS * head_dim if kv_page_stride is None else kv_page_stride
    _check_slots(slots, out.shape[0])
    _check_pool(kv_pages, None, num_pages, 2 * PAGE_POSITIONS * head_dim, kv_page_stride, 0)
    dev = _device_of((("out", out), ("slots", slots), ("kv_pages", kv_pages)))
    return _launch("idx_load_slots_bf16", dev, stream, check, _addr(kv_pages), _addr(slots), out.shape[0], head_dim,
                   num_pages, kv_page_stride, _addr(out), _row_stride(out))


def idx_latent_attention_workspace(rows, num_heads, table_width, k=None) -> int:
    """Bytes of workspace that a latent attention call of these sizes needs on
    the current device (``k`` None: no selection)."""
    return int(_lib.idx_latent_attention_workspace(rows, num_heads, table_width, -1 if k is None else k))


def _latent_workspace(rows, heads, width, k, dev, stream) -> torch.Tensor | None:
    """A workspace from torch's allocator, on the call's device and stream."""
    if dev is None:
        return None
    with torch.cuda.device(dev):
        need = idx_latent_attention_workspace(rows, heads, width, k)
        if need <= 0:
            return None
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=dev)
        if not isinstance(stream, torch.cuda.Stream):
            raise ValueError("a call on a raw stream handle needs its own workspace")
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=dev)


def _latent_attention(name, q, kv_pages, kscale, page_table, topk_idx, seqlens, out, lse, scale, num_pages, sinks,
                      row_table, workspace, strides, page_table_row_stride, stream, check):
    """``kscale`` and ``strides`` are tuples: those of the pool's key type."""
    _check("q", q, torch.bfloat16)
    _check("out", out, torch.bfloat16)
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError(f"q and out must be [rows, heads, {LATENT_DIM}], got {list(q.shape)} and {list(out.shape)}")
    rows, heads, head_dim = q.shape
    _check("page_table", page_table, torch.int32, dense_rows=True)
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dims")
    tables, width = page_table.shape
    for what, x, dtype, shape in (("seqlens", seqlens, torch.int32, (rows,)), ("sinks", sinks, torch.float32, (heads,)),
                                  ("lse", lse, torch.float32, (rows, heads)), ("row_table", row_table, torch.int32, (rows,))):
        if x is not None:
            _check(what, x, dtype)
            if x.shape != shape:
                raise ValueError(f"{what} must be {list(shape)}, got {list(x.shape)}")
    k = None
    if topk_idx is not None:
        _check("topk_idx", topk_idx, torch.int32)
        if topk_idx.dim() != 2 or topk_idx.shape[0] != rows:
            raise ValueError(f"topk_idx must be [{rows}, k], got {list(topk_idx.shape)}")
        k = topk_idx.shape[1]
    if page_table_row_stride is None:
        shared = tables == 1 and row_table is None
        page_table_row_stride = 0 if shared else page_table.stride(0)
        if not shared and row_table is None and tables < rows:
            raise ValueError(f"page_table holds {tables} tables for {rows} rows")
    _check_pool(kv_pages, kscale[0] if kscale else None, num_pages,
                PAGE_POSITIONS * LATENT_DIM * (1 if kscale else 2), strides[0], strides[-1])
    dev = _device_of((("q", q), ("kv_pages", kv_pages), ("kscale", kscale[0] if kscale else None),
                      ("page_table", page_table), ("topk_idx", topk_idx), ("seqlens", seqlens), ("out", out),
                      ("lse", lse), ("sinks", sinks), ("row_table", row_table), ("workspace", workspace)))
    if workspace is None:
        workspace = _latent_workspace(rows, heads, width, k, dev, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _launch(name, dev, stream, check, _addr(q), _addr(kv_pages), *[_addr(x) for x in kscale], _addr(page_table),
                   _addr(row_table), 0 if row_table is None else tables, _addr(topk_idx), _addr(seqlens), _addr(sinks),
                   _addr(out), _addr(lse), rows, heads, head_dim, width, num_pages, *strides, page_table_row_stride,
                   -1 if k is None else k, scale, _addr(workspace), nbytes)


def idx_latent_attention_fp8(q, kv_pages, kscale, page_table, topk_idx, seqlens, out, lse=None, *, scale, num_pages,
                             sinks=None, row_table=None, workspace=None,
                             kv_page_stride=PAGE_POSITIONS * (LATENT_DIM + 4),
                             kscale_page_stride=PAGE_POSITIONS * (LATENT_DIM + 4), page_table_row_stride=None,
                             stream=None, check=True) -> int:
    """Attention of bf16 ``q`` [rows, heads, 512] to the fp8 latents of the positions
    in ``topk_idx`` (int32 [rows, k], as the top-k leaves it; None: every position
    below ``seqlens``), which are key and value of all heads; into ``out`` (as
    ``q``) and, if given, ``lse`` fp32 [rows, heads].

    ``page_table`` int32 [tables, width]: one for all rows, one per row, or row b's
    at ``row_table[b]``.  ``sinks`` fp32 [heads] join the softmax's denominator.
    ``workspace``: a tensor of :func:`idx_latent_attention_workspace` bytes, of this
    call's own while it runs; None takes one from torch's allocator.
    """
    return _latent_attention("idx_latent_attention_fp8", q, kv_pages, (kscale,), page_table, topk_idx, seqlens, out,
                             lse, scale, num_pages, sinks, row_table, workspace, (kv_page_stride, kscale_page_stride),
                             page_table_row_stride, stream, check)


def idx_latent_attention_bf16(q, kv_pages, page_table, topk_idx, seqlens, out, lse=None, *, scale, num_pages,
                              sinks=None, row_table=None, workspace=None,
                              kv_page_stride=2 * PAGE_POSITIONS * LATENT_DIM, page_table_row_stride=None, stream=None,
                              check=True) -> int:
    """bf16 counterpart of :func:`idx_latent_attention_fp8`."""
    return _latent_attention("idx_latent_attention_bf16", q, kv_pages, (), page_table, topk_idx, seqlens, out, lse,
                             scale, num_pages, sinks, row_table, workspace, (kv_page_stride,), page_table_row_stride,
                             stream, check)


__all__ = [
    "idx_paged_mqa_logits_fp8", "idx_paged_mqa_logits_bf16", "idx_paged_mqa_logits_varlen_fp8",
    "idx_paged_mqa_logits_varlen_bf16", "idx_topk_logits",
    "idx_paged_mqa_topk_fp8", "idx_paged_mqa_topk_bf16", "idx_store_keys_fp8",
    "idx_store_keys_bf16", "idx_status_string",
    "idx_norm_rope", "idx_norm_rope_store_fp8", "idx_norm_rope_store_bf16",
    "idx_load_slots_fp8", "idx_load_slots_bf16",
    "idx_latent_attention_fp8", "idx_latent_attention_bf16", "idx_latent_attention_workspace",
    "idx_abi_version", "IdxError", "LIB_PATH", "NUM_HEADS", "HEAD_DIM", "PAGE_POSITIONS", "LATENT_DIM",
]
