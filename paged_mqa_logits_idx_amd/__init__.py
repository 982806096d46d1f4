"""Python binding of the paged MQA-logits indexer library (libidx_paged_mqa.so).

Argument marshalling only: every step of the computation runs in the library's
HIP kernels (the marshalling of the newer functions is compiled, csrc/binding.cpp).
The functions carry the C-ABI names and argument order; they
accept torch device tensors (or raw device addresses as ints, but for the
compiled ones) and pass their addresses and sizes through ctypes.  torch supplies
device memory and streams.

The library must be built in-tree first (``python paged_mqa_logits_idx_amd/_build.py``
or ``__graft_entry__.build()``); importing this module without it raises.  Where the
compiled marshalling does not load, the functions that use it raise when called.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch  # loads the HIP runtime the library binds to (same soname)


class _Missing:
    """In the place of the compiled marshalling where it does not load (not built, or
    built for another Python or torch): its calls say so, the others do without it."""

    def __init__(self, error):
        self._error = error

    def __getattr__(self, name):
        raise ImportError(f"{Path(__file__).resolve().parent / '_binding.so'}: {self._error}; build it first "
                          "(python paged_mqa_logits_idx_amd/_build.py)") from self._error


try:
    from . import _binding  # compiled with the library
except ImportError as e:
    _binding = _Missing(e)

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
    "idx_plan_batch",
    "idx_store_kv_fp8",
    "idx_store_kv_bf16",
    "idx_page_bounds_fp8",
    "idx_page_bounds_bf16",
    "idx_page_scores",
    "idx_kv_attention_fp8",
    "idx_kv_attention_bf16",
    "idx_kv_attention_workspace",
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
             + [i32, ctypes.c_float, ptr, i64, ptr]),
            ("idx_plan_batch", [ptr, ptr, i32, ptr, i64, ptr, i32, i64, i64] + [ptr] * 7),
            ("idx_store_kv_fp8", [ptr] * 3 + [i64, i32, i32, i64, i64] + [ptr] * 4 + [i64] * 5 + [ptr]),
            ("idx_store_kv_bf16", [ptr] * 3 + [i64, i32, i32, i64, i64] + [ptr] * 2 + [i64] * 3 + [ptr]),
            ("idx_page_bounds_fp8", [ptr] * 4 + [i32] + [ptr] * 3 + [i32] * 4 + [i64] * 6 + [ptr]),
            ("idx_page_bounds_bf16", [ptr] * 3 + [i32] + [ptr] * 3 + [i32] * 4 + [i64] * 4 + [ptr]),
            ("idx_page_scores", [ptr] * 4 + [i32] + [ptr] * 3 + [i32] * 5 + [i64] * 3 + [i32, i32, ptr]),
            ("idx_kv_attention_fp8", [ptr] * 7 + [i32] + [ptr] * 5 + [i32] * 5 + [i64] * 6
             + [i32, ctypes.c_float, ptr, i64, ptr]),
            ("idx_kv_attention_bf16", [ptr] * 5 + [i32] + [ptr] * 5 + [i32] * 5 + [i64] * 4
             + [i32, ctypes.c_float, ptr, i64, ptr])):
        fn = getattr(lib, name)
        fn.argtypes = types
        fn.restype = ctypes.c_int
    lib.idx_latent_attention_workspace.argtypes = [i32] * 4
    lib.idx_latent_attention_workspace.restype = i64
    lib.idx_kv_attention_workspace.argtypes = [i32] * 6
    lib.idx_kv_attention_workspace.restype = i64
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


# --- the latent cache's operators (include/latent_cache.h).  Their arguments are
# tensors; a call on a few tokens takes the GPU a few microseconds, so the checks
# below stay short: dtype, shape, layout and device of each, once.

# (the public current_stream builds an object, which takes half as long as a
# launch, and the public current_device looks whether the runtime has started)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _elsewhere(name, x, dev) -> ValueError:
    return ValueError(f"{name} is on {x.device}, the arguments before it on " + ("cpu" if dev < 0 else f"cuda:{dev}"))


def _dense(name, x, dtype, shape, dev) -> int:
    """Address of a contiguous tensor of this type and shape on device ``dev``."""
    if x.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if x.get_device() != dev:
        raise _elsewhere(name, x, dev)
    return x.data_ptr()


def _rows(name, x, dims) -> int:
    """Elements between the rows (first dim) of a bf16 tensor of ``dims`` dims
    whose rows are dense."""
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {x.dtype}")
    shape = x.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dims, got {list(shape)}")
    if x.is_contiguous():
        return shape[1] if dims == 2 else shape[1] * shape[2]
    dense = 1
    for size, step in zip(reversed(shape[1:]), reversed(x.stride()[1:])):
        if size > 1 and step != dense:
            raise ValueError(f"{name} must be dense behind its first dim")
        dense *= size
    return x.stride(0) if shape[0] > 1 else dense


# Where the library's text names the indexer's sizes.
_STATUS_TEXT = {IDX_ERR_UNSUPPORTED: "unsupported num_heads, head_dim, rope_dim or flag"}


def _launch(fn, dev, stream, check, *args) -> int:
    """Calls the library on the tensors' device, whatever the current one is."""
    if dev < 0:
        raise ValueError("tensors passed to the indexer library must be device tensors")
    handle = _raw_stream(dev) if stream is None else _stream_handle(stream, dev)
    if dev == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if check and status != IDX_OK:
        raise IdxError(status, f"{fn.__name__}: {_STATUS_TEXT.get(status) or idx_status_string(status)}")
    return status


def _rotation(x, dev, positions, inv_freq, weight, norm, leading, halves):
    """The norm and rotation's arguments: addresses of weight, positions and
    inv_freq, rope_dim and flags."""
    shape = x.shape
    flags = (0 if norm else IDX_NORM_OFF) | (IDX_ROPE_LEADING if leading else 0) | (IDX_ROPE_HALVES if halves else 0)
    w = p = f = None
    rope = 0
    if weight is not None:
        if not norm:
            raise ValueError("weight goes with the norm")
        w = _dense("weight", weight, torch.float32, shape[-1:], dev)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    if positions is not None:
        p = _dense("positions", positions, torch.int64, shape[:1], dev)
        rope = 2 * inv_freq.numel()
        f = _dense("inv_freq", inv_freq, torch.float32, (rope // 2,), dev)
    return w, p, f, rope, flags


def _pool(kv_pages, kscale, num_pages, page_bytes, kv_page_stride, kscale_page_stride, dev):
    """Addresses of a pool and its scales, which as tensors must hold the pages
    (``page_bytes`` of values each) that they are said to hold."""
    kv, ks = kv_pages, kscale
    if isinstance(kv_pages, torch.Tensor):
        if not kv_pages.is_contiguous():
            raise ValueError("kv_pages must be contiguous")
        if num_pages > 0 and kv_pages.nbytes < (num_pages - 1) * kv_page_stride + page_bytes:
            raise ValueError(f"kv_pages is shorter than {num_pages} pages of {kv_page_stride} bytes")
        if kv_pages.get_device() != dev:
            raise _elsewhere("kv_pages", kv_pages, dev)
        kv = kv_pages.data_ptr()
    if isinstance(kscale, torch.Tensor):
        if kscale.dtype is not torch.float32:
            raise ValueError(f"kscale must be torch.float32, got {kscale.dtype}")
        if not kscale.is_contiguous():
            raise ValueError("kscale must be contiguous")
        if num_pages > 0 and kscale.nbytes < (num_pages - 1) * kscale_page_stride + 4 * PAGE_POSITIONS:
            raise ValueError(f"kscale is shorter than {num_pages} pages of {kscale_page_stride} bytes")
        if kscale.get_device() != dev:
            raise _elsewhere("kscale", kscale, dev)
        ks = kscale.data_ptr()
    return kv, ks


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
    stride, dev = _rows("x", x, 3), x.get_device()
    n, heads, dim = x.shape
    to = _dense("out", out, torch.bfloat16, x.shape, dev)
    w, p, f, rope, flags = _rotation(x, dev, positions, inv_freq, weight, norm, leading, halves)
    return _launch(_lib.idx_norm_rope, dev, stream, check, x.data_ptr(), w, p, f, to, n, heads, dim, rope, flags, eps,
                   stride)


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
    stride, dev = _rows("x", x, 2), x.get_device()
    n, dim = x.shape
    fused = PAGE_POSITIONS * (dim + 4)
    kv_page_stride = fused if kv_page_stride is None else kv_page_stride
    kscale_page_stride = fused if kscale_page_stride is None else kscale_page_stride
    w, p, f, rope, flags = _rotation(x, dev, positions, inv_freq, weight, norm, leading, halves)
    at = _dense("slots", slots, torch.int64, (n,), dev)
    kv, ks = _pool(kv_pages, kscale, num_pages, PAGE_POSITIONS * dim, kv_page_stride, kscale_page_stride, dev)
    return _launch(_lib.idx_norm_rope_store_fp8, dev, stream, check, x.data_ptr(), w, p, f, at, n, dim, rope, flags, eps,
                   stride, kv, ks, num_pages, kv_page_stride, kscale_page_stride)


def idx_norm_rope_store_bf16(x, positions, inv_freq, slots, kv_pages, *, num_pages, weight=None, eps=1e-6,
                             norm=True, leading=False, halves=False, kv_page_stride=None, stream=None,
                             check=True) -> int:
    """bf16 counterpart of :func:`idx_norm_rope_store_fp8`: pages of 128*D bytes."""
    stride, dev = _rows("x", x, 2), x.get_device()
    n, dim = x.shape
    page = 2 * PAGE_POSITIONS * dim
    kv_page_stride = page if kv_page_stride is None else kv_page_stride
    w, p, f, rope, flags = _rotation(x, dev, positions, inv_freq, weight, norm, leading, halves)
    at = _dense("slots", slots, torch.int64, (n,), dev)
    kv, _ = _pool(kv_pages, None, num_pages, page, kv_page_stride, 0, dev)
    return _launch(_lib.idx_norm_rope_store_bf16, dev, stream, check, x.data_ptr(), w, p, f, at, n, dim, rope, flags, eps,
                   stride, kv, num_pages, kv_page_stride)


def idx_load_slots_fp8(kv_pages, kscale, slots, out, *, num_pages, kv_page_stride=None,
                       kscale_page_stride=None, stream=None, check=True) -> int:
    """out[t] = bf16(code * scale) of pool slot slots[t], for bf16 ``out`` [n, D]
    (D 128 or 512; rows may be strided).  A slot out of range leaves its row."""
    stride, dev = _rows("out", out, 2), out.get_device()
    n, dim = out.shape
    fused = PAGE_POSITIONS * (dim + 4)
    kv_page_stride = fused if kv_page_stride is None else kv_page_stride
    kscale_page_stride = fused if kscale_page_stride is None else kscale_page_stride
    at = _dense("slots", slots, torch.int64, (n,), dev)
    kv, ks = _pool(kv_pages, kscale, num_pages, PAGE_POSITIONS * dim, kv_page_stride, kscale_page_stride, dev)
    return _launch(_lib.idx_load_slots_fp8, dev, stream, check, kv, ks, at, n, dim, num_pages, kv_page_stride,
                   kscale_page_stride, out.data_ptr(), stride)


def idx_load_slots_bf16(kv_pages, slots, out, *, num_pages, kv_page_stride=None, stream=None, check=True) -> int:
    """bf16 counterpart of :func:`idx_load_slots_fp8`."""
    stride, dev = _rows("out", out, 2), out.get_device()
    n, dim = out.shape
    page = 2 * PAGE_POSITIONS * dim
    kv_page_stride = page if kv_page_stride is None else kv_page_stride
    at = _dense("slots", slots, torch.int64, (n,), dev)
    kv, _ = _pool(kv_pages, None, num_pages, page, kv_page_stride, 0, dev)
    return _launch(_lib.idx_load_slots_bf16, dev, stream, check, kv, at, n, dim, num_pages, kv_page_stride,
                   out.data_ptr(), stride)


def idx_latent_attention_workspace(rows, num_heads, table_width, k=None) -> int:
    """Bytes of workspace that a latent attention call of these sizes needs on
    the current device (``k`` None: no selection)."""
    return _lib.idx_latent_attention_workspace(rows, num_heads, table_width, -1 if k is None else k)


def _workspace(size, dims, dev, stream) -> torch.Tensor | None:
    """A workspace of ``size(*dims)`` bytes from torch's allocator, on the call's
    device and stream."""
    if dev < 0:
        return None
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _workspace(size, dims, dev, stream)
    need = size(*dims)
    if need <= 0:
        return None
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device="cuda")
    if not isinstance(stream, torch.cuda.Stream):
        raise ValueError("a call on a raw stream handle needs its own workspace")
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device="cuda")


def _latent_attention(fn, q, kv_pages, kscale, page_table, topk_idx, seqlens, out, lse, scale, num_pages, sinks,
                      row_table, workspace, strides, page_table_row_stride, stream, check):
    """``kscale`` and ``strides`` are tuples: those of the pool's key type."""
    dev, shape = q.get_device(), q.shape
    if len(shape) != 3 or out.shape != shape:
        raise ValueError(f"q and out must be [rows, heads, {LATENT_DIM}], got {list(shape)} and {list(out.shape)}")
    rows, heads, dim = shape
    from_q = _dense("q", q, torch.bfloat16, shape, dev)
    to = _dense("out", out, torch.bfloat16, shape, dev)
    if page_table.dtype is not torch.int32:
        raise ValueError(f"page_table must be torch.int32, got {page_table.dtype}")
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dims")
    tables, width = page_table.shape
    step, unit = page_table.stride()
    if unit != 1 and width > 1:
        raise ValueError("page_table must be unit-stride along its last dim")
    if page_table.get_device() != dev:
        raise _elsewhere("page_table", page_table, dev)
    lengths = _dense("seqlens", seqlens, torch.int32, (rows,), dev)
    idx = sink = log = which = None
    k = -1
    if topk_idx is not None:
        if topk_idx.dim() != 2 or topk_idx.shape[0] != rows:
            raise ValueError(f"topk_idx must be [{rows}, k], got {list(topk_idx.shape)}")
        k = topk_idx.shape[1]
        idx = _dense("topk_idx", topk_idx, torch.int32, (rows, k), dev)
    if sinks is not None:
        sink = _dense("sinks", sinks, torch.float32, (heads,), dev)
    if lse is not None:
        log = _dense("lse", lse, torch.float32, (rows, heads), dev)
    if row_table is not None:
        which = _dense("row_table", row_table, torch.int32, (rows,), dev)
    if page_table_row_stride is None:
        shared = tables == 1 and row_table is None
        page_table_row_stride = 0 if shared else step
        if not shared and row_table is None and tables < rows:
            raise ValueError(f"page_table holds {tables} tables for {rows} rows")
    kv, *ks = _pool(kv_pages, kscale[0] if kscale else None, num_pages,
                    PAGE_POSITIONS * LATENT_DIM * (1 if kscale else 2), strides[0], strides[-1], dev)
    if workspace is None:
        workspace = _workspace(_lib.idx_latent_attention_workspace, (rows, heads, width, k), dev, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    elif workspace.get_device() != dev:
        raise _elsewhere("workspace", workspace, dev)
    space, nbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    return _launch(fn, dev, stream, check, from_q, kv, *(ks if kscale else ()), page_table.data_ptr(), which,
                   0 if which is None else tables, idx, lengths, sink, to, log, rows, heads, dim, width, num_pages,
                   *strides, page_table_row_stride, k, scale, space, nbytes)


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
    return _latent_attention(_lib.idx_latent_attention_fp8, q, kv_pages, (kscale,), page_table, topk_idx, seqlens, out,
                             lse, scale, num_pages, sinks, row_table, workspace, (kv_page_stride, kscale_page_stride),
                             page_table_row_stride, stream, check)


def idx_latent_attention_bf16(q, kv_pages, page_table, topk_idx, seqlens, out, lse=None, *, scale, num_pages,
                              sinks=None, row_table=None, workspace=None,
                              kv_page_stride=2 * PAGE_POSITIONS * LATENT_DIM, page_table_row_stride=None, stream=None,
                              check=True) -> int:
    """bf16 counterpart of :func:`idx_latent_attention_fp8`."""
    return _latent_attention(_lib.idx_latent_attention_bf16, q, kv_pages, (), page_table, topk_idx, seqlens, out, lse,
                             scale, num_pages, sinks, row_table, workspace, (kv_page_stride,), page_table_row_stride,
                             stream, check)


# --- the cache of keys and values by head (include/kv_cache.h).  Its pools are
# tensors [pages, kv_heads, 64, D], whose strides the kernels take.  The marshalling
# of these calls is compiled (csrc/binding.cpp).


def _make_workspace(nbytes, stream) -> torch.Tensor:
    """A workspace from torch's allocator on a stream that is not the current one."""
    if not isinstance(stream, torch.cuda.Stream):
        raise ValueError("a call on a raw stream handle needs its own workspace")
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


if not isinstance(_binding, _Missing):
    _binding.bind(_make_workspace, *(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in (
        "idx_plan_batch", "idx_store_kv_fp8", "idx_store_kv_bf16", "idx_page_bounds_fp8", "idx_page_bounds_bf16",
        "idx_page_scores", "idx_kv_attention_fp8", "idx_kv_attention_bf16", "idx_kv_attention_workspace")))


def _done(name, status, check) -> int:
    """The status of a call, raised where it is an error and ``check``."""
    if check and status != IDX_OK:
        raise IdxError(status, f"{name}: {_STATUS_TEXT.get(status) or idx_status_string(status)}")
    return status


def idx_plan_batch(cached, added, free_pages, page_table, slots=None, positions=None, row_table=None, seqlens=None,
                   starts=None, taken=None, *, stream=None, check=True) -> int:
    """Page tables and slot maps of a step, from its requests' lengths.

    Request r holds ``cached[r]`` positions (int32) and gets ``added[r]`` more; the
    pages it lacks come from ``free_pages`` (int32, in order, request by request)
    into its row of ``page_table`` (int32 [requests, width]).  Its new tokens are
    rows of the batch, request by request: ``slots`` and ``positions`` int64 [n],
    ``row_table`` and ``seqlens`` int32 [n] (rows past the last token: slot -1,
    length 0), ``starts`` int64 [requests + 1] each request's first row, ``taken``
    int64 [1] the pages asked for.  Those that are None are not written.
    """
    status = _binding.plan_batch(cached, added, free_pages, page_table, slots, positions, row_table, seqlens, starts, taken,
                                 stream)
    return status and _done("idx_plan_batch", status, check)


def idx_store_kv_fp8(keys, values, slots, k_pages, v_pages, kscale, vscale, *, num_pages=None, stream=None,
                     check=True) -> int:
    """Quantise bf16 ``keys`` and ``values`` [n, kv_heads, D] (D 64, 128 or 256; first
    dims may be strided), vector by vector (scale = amax/448, e4m3fn codes), into pool
    slots.

    ``k_pages`` and ``v_pages``: uint8 or float8_e4m3fn [pages, kv_heads, 64, D], of the
    same strides, dense behind the first two dims; ``kscale`` and ``vscale``: fp32 [pages,
    kv_heads, 64] likewise.  ``slots`` int64 [n] (64*page + position; out of range skips
    the token).
    """
    status = _binding.store_kv(True, keys, values, slots, k_pages, v_pages, kscale, vscale, num_pages, stream)
    return status and _done("idx_store_kv_fp8", status, check)


def idx_store_kv_bf16(keys, values, slots, k_pages, v_pages, *, num_pages=None, stream=None, check=True) -> int:
    """bf16 counterpart of :func:`idx_store_kv_fp8`: a copy."""
    status = _binding.store_kv(False, keys, values, slots, k_pages, v_pages, None, None, num_pages, stream)
    return status and _done("idx_store_kv_bf16", status, check)


def idx_page_bounds_fp8(k_pages, kscale, page_table, seqlens, bounds, *, first=None, row_table=None, num_pages=None,
                        stream=None, check=True) -> int:
    """Least and largest value of each dim of the keys in pages: for row b the pages of
    its positions from ``first[b]`` (int32 [rows]; None: 0) to ``seqlens[b]``, into bf16
    ``bounds`` [pages, kv_heads, 2, D], rounded outwards.

    Pools as in :func:`idx_store_kv_fp8`, ``page_table`` int32 [tables, width]: one for
    all rows, one per row, or row b's at ``row_table[b]``.
    """
    status = _binding.page_bounds(True, k_pages, kscale, page_table, seqlens, bounds, first, row_table, num_pages,
                                  stream)
    return status and _done("idx_page_bounds_fp8", status, check)


def idx_page_bounds_bf16(k_pages, page_table, seqlens, bounds, *, first=None, row_table=None, num_pages=None, stream=None,
                         check=True) -> int:
    """bf16 counterpart of :func:`idx_page_bounds_fp8`."""
    status = _binding.page_bounds(False, k_pages, None, page_table, seqlens, bounds, first, row_table, num_pages,
                                  stream)
    return status and _done("idx_page_bounds_bf16", status, check)


def idx_page_scores(q, bounds, page_table, seqlens, scores, page_counts=None, *, first_pages=0, last_pages=0,
                    row_table=None, stream=None, check=True) -> int:
    """The most that any key within a page's ``bounds`` (bf16 [pages, kv_heads, 2, D])
    could score with the query heads of bf16 ``q`` [rows, heads, D] that share a key
    head, into ``scores`` fp32 [rows, kv_heads, width] (rows may be strided); +inf for
    a row's first and last pages, -inf past them.  ``page_counts`` int32 [rows,
    kv_heads]: live pages.

    ``scores.flatten(0, 1)`` and ``page_counts.flatten()`` are what
    :func:`idx_topk_logits` selects pages from (score rows a multiple of 4 apart).
    """
    status = _binding.page_scores(q, bounds, page_table, seqlens, scores, page_counts, first_pages, last_pages, row_table,
                                  stream)
    return status and _done("idx_page_scores", status, check)


def idx_kv_attention_workspace(rows, num_heads, kv_heads, head_dim, table_width, k=None) -> int:
    """Bytes of workspace that a call of :func:`idx_kv_attention_fp8` or its counterpart
    of these sizes needs on the current device (``k`` None: no selection)."""
    return _lib.idx_kv_attention_workspace(rows, num_heads, kv_heads, head_dim, table_width, -1 if k is None else k)


def idx_kv_attention_fp8(q, k_pages, v_pages, kscale, vscale, page_table, page_idx, seqlens, out, lse=None, *, scale,
                         sinks=None, row_table=None, workspace=None, num_pages=None, stream=None, check=True) -> int:
    """Attention of bf16 ``q`` [rows, heads, D], one new token a row, to the fp8 keys and
    values of its pages (pools as in :func:`idx_store_kv_fp8`; heads / kv_heads query
    heads share a key head) into ``out`` (as ``q``) and, if given, ``lse`` fp32 [rows,
    heads].

    ``page_idx`` int32 [rows, kv_heads, k] (or [rows * kv_heads, k]): the pages to attend
    to, as the top-k leaves them; None: all below ``seqlens``.  ``page_table`` int32
    [tables, width]: one for all rows, one per row, or row b's at ``row_table[b]``.
    ``sinks`` fp32 [heads] join the softmax's denominator.  ``workspace``: a tensor of
    :func:`idx_kv_attention_workspace` bytes, of this call's own while it runs; None takes
    one from torch's allocator.
    """
    status = _binding.kv_attention(True, q, k_pages, v_pages, kscale, vscale, page_table, page_idx, seqlens, out, lse, scale,
                                   sinks, row_table, workspace, num_pages, stream)
    return status and _done("idx_kv_attention_fp8", status, check)


def idx_kv_attention_bf16(q, k_pages, v_pages, page_table, page_idx, seqlens, out, lse=None, *, scale, sinks=None,
                          row_table=None, workspace=None, num_pages=None, stream=None, check=True) -> int:
    """bf16 counterpart of :func:`idx_kv_attention_fp8`."""
    status = _binding.kv_attention(False, q, k_pages, v_pages, None, None, page_table, page_idx, seqlens, out, lse, scale,
                                   sinks, row_table, workspace, num_pages, stream)
    return status and _done("idx_kv_attention_bf16", status, check)


__all__ = [
    "idx_paged_mqa_logits_fp8", "idx_paged_mqa_logits_bf16", "idx_paged_mqa_logits_varlen_fp8",
    "idx_paged_mqa_logits_varlen_bf16", "idx_topk_logits",
    "idx_paged_mqa_topk_fp8", "idx_paged_mqa_topk_bf16", "idx_store_keys_fp8",
    "idx_store_keys_bf16", "idx_status_string",
    "idx_norm_rope", "idx_norm_rope_store_fp8", "idx_norm_rope_store_bf16",
    "idx_load_slots_fp8", "idx_load_slots_bf16",
    "idx_latent_attention_fp8", "idx_latent_attention_bf16", "idx_latent_attention_workspace",
    "idx_plan_batch", "idx_store_kv_fp8", "idx_store_kv_bf16", "idx_page_bounds_fp8", "idx_page_bounds_bf16",
    "idx_page_scores", "idx_kv_attention_fp8", "idx_kv_attention_bf16", "idx_kv_attention_workspace",
    "idx_abi_version", "IdxError", "LIB_PATH", "NUM_HEADS", "HEAD_DIM", "PAGE_POSITIONS", "LATENT_DIM",
]
