"""Paged MLA decode for GB300 (sm_103a): Python binding of the C ABI.

The compute path lives in ``_lib/libmla_gb300.so`` (built from ``csrc/`` by
``mla_latent_kv_cache_gb300.build``). This module only marshals arguments:
torch tensors -> device pointers, the current CUDA stream, and status codes ->
exceptions. Before a call it checks what the library cannot see (that every
tensor is a CUDA tensor on one device, and the dtypes, layouts and sizes of
the buffers the call reads and writes) and raises MlaError with
MLA_ERR_INVALID_ARG otherwise. There is no fallback: if the library is
missing, every call raises.

Entry points mirror ``include/mla.h``:
  mla_cache_write, mla_decode_workspace_bytes, mla_decode, mla_decode_varlen,
  mla_merge_lse, mla_gather_upconvert, mla_cache_write_latent,
  mla_decode_latent_workspace_bytes, mla_decode_latent,
  mla_decode_static_scratch (+ mla_static_scratch_status), mla_prefill,
  mla_attn_weights, mla_cache_evict, mla_num_sms, mla_row_bytes,
  mla_status_string.
``decode(...)`` is a convenience wrapper that allocates the outputs and the
workspace with torch and calls ``mla_decode``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmla_gb300.so")

MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_WORKSPACE, MLA_ERR_CUDA = 0, -1, -2, -3, -4
MLA_CACHE_BF16_576, MLA_CACHE_FP8_DS_MLA_656 = 0, 1
MLA_OUT_BF16, MLA_OUT_F32 = 0, 1
STATUS_WAIT_TIMEOUT, STATUS_BAD_BLOCK = 1, 2

_lock = threading.Lock()
_lib = None


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {mla_status_string(status)} ({status})" + (f": {detail}" if detail else ""))


def load() -> ctypes.CDLL:
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build it with `python -m mla_latent_kv_cache_gb300.build` "
                    "(there is no CPU fallback)")
            lib = ctypes.CDLL(LIB_PATH)
            vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
            lib.mla_row_bytes.argtypes = [i32]
            lib.mla_row_bytes.restype = i32
            lib.mla_status_string.argtypes = [i32]
            lib.mla_status_string.restype = ctypes.c_char_p
            lib.mla_num_sms.argtypes = []
            lib.mla_num_sms.restype = i32
            lib.mla_cache_write.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, vp]
            lib.mla_cache_write.restype = i32
            lib.mla_decode_workspace_bytes.argtypes = [i32, i32, i32, i32]
            lib.mla_decode_workspace_bytes.restype = sz
            lib.mla_decode.argtypes = [vp, vp, vp, i32, i64, i32, vp, i64, vp, i32, i32, i32, f32, vp, i32, vp,
                                       vp, sz, i32, vp]
            lib.mla_decode.restype = i32
            lib.mla_decode_static_scratch.argtypes = [vp, vp, vp, i32, i64, i32, vp, i64, vp, i32, i32, i32, f32, vp,
                                                      i32, vp, i32, vp]
            lib.mla_decode_static_scratch.restype = i32
            lib.mla_static_scratch_status.argtypes = [vp, i32, vp]
            lib.mla_static_scratch_status.restype = i32
            lib.mla_test_hold_next_decode.argtypes = []
            lib.mla_test_hold_next_decode.restype = None
            lib.mla_test_slow_pv_next_decode.argtypes = []
            lib.mla_test_slow_pv_next_decode.restype = None
            lib.mla_test_limit_next_evict.argtypes = [i32]
            lib.mla_test_limit_next_evict.restype = None
            lib.mla_merge_lse.argtypes = [vp, vp, i32, i64, vp, i32, vp, vp]
            lib.mla_decode_varlen.argtypes = [vp, vp, i64, vp, i32, i64, i32, vp, i64, vp, vp, i32, i32, i32, f32,
                                              vp, i32, vp, vp, ctypes.c_size_t, i32, vp]
            lib.mla_decode_varlen.restype = i32
            lib.mla_gather_upconvert.argtypes = [vp, i64, i32, vp, i64, vp, i32, i64, vp, i64, vp]
            lib.mla_gather_upconvert.restype = i32
            lib.mla_cache_write_latent.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, vp]
            lib.mla_cache_write_latent.restype = i32
            lib.mla_decode_latent_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            lib.mla_decode_latent_workspace_bytes.restype = sz
            lib.mla_decode_latent.argtypes = [vp, vp, vp, i32, i64, i32, vp, i64, vp, i32, i32, i32, f32, vp, i32,
                                              vp, vp, sz, i32, vp]
            lib.mla_decode_latent.restype = i32
            lib.mla_merge_lse.restype = i32
            lib.mla_prefill.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, i32, i64, i64, i32,
                                        i32, i32, i32, f32, vp, vp, vp, vp]
            lib.mla_prefill.restype = i32
            lib.mla_attn_weights.argtypes = [vp, vp, vp, vp, i32, i32, i64, i32, vp, i64, vp, i32, i32, i32, f32, f32,
                                             vp, i64, i32, vp, i32, vp]
            lib.mla_attn_weights.restype = i32
            lib.mla_cache_evict.argtypes = [vp, i32, i64, i32, vp, i64, vp, vp, vp, i64, i32, vp, i32, i32, i32, vp,
                                            vp, vp, vp, i64, vp, vp]
            lib.mla_cache_evict.restype = i32
            _lib = lib
    return _lib


# the current stream's handle without a Stream object around it (a few microseconds a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str) -> None:
    if status != MLA_OK:
        raise MlaError(status, where)


# Argument checks of the binding. The library validates sizes, pointers and
# alignment on the host, but it cannot tell a host pointer from a device one
# or how large a caller's buffer is: a host tensor handed to a kernel is an
# illegal address (or, where the GPU reaches host memory, a silent slow
# path), and an output smaller than the call writes is overrun. These checks
# run before the library is called and raise MlaError(MLA_ERR_INVALID_ARG).

def _is_cuda(t) -> bool:
    return isinstance(t, torch.Tensor) and t.is_cuda


def _need(ok: bool, where: str, detail: str) -> None:
    if not ok:
        raise MlaError(MLA_ERR_INVALID_ARG, where, detail)


def _on_device(where: str, **tensors) -> None:
    """Every tensor passed as a device pointer is a CUDA tensor, all on one device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        _need(_is_cuda(t), where, f"{name} must be a CUDA tensor")
        if dev is None:
            dev = t.device
        _need(t.device == dev, where, f"{name} is on {t.device}, the other arguments on {dev}")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _table_stride(block_table) -> int:
    """A table's row stride for the library, which takes it as a row's length.
    torch leaves the stride of a dimension of one entry as it comes (a [P, 1]
    table transposed to [1, P] has strides (1, 1)), so a single row is at least
    as long as its columns."""
    rows, cols = block_table.shape
    return max(block_table.stride(0), cols) if rows == 1 else block_table.stride(0)


def _decode_args(where, q_lat, q_pe, cache, block_table, seq_lens, out, lse, workspace, rows, width):
    """Checks shared by the decode entry points: `rows` query rows of `width`
    latent values (query tokens x heads)."""
    _on_device(where, q_lat=q_lat, q_pe=q_pe, cache=cache, block_table=block_table, seq_lens=seq_lens, out=out,
               lse=lse, workspace=workspace)
    _need(q_lat.dtype == torch.bfloat16 and q_pe.dtype == torch.bfloat16, where, "q_lat and q_pe must be bf16")
    _need(q_lat.is_contiguous() and q_pe.is_contiguous(), where, "q_lat and q_pe must be contiguous")
    _need(q_lat.numel() == rows * width and q_pe.numel() == rows * 64, where,
          f"q_lat / q_pe hold {q_lat.numel()} / {q_pe.numel()} values, {rows} rows of {width} / 64 expected")
    _need(out.dtype in (torch.bfloat16, torch.float32) and out.is_contiguous(), where,
          "out must be a contiguous bf16 or fp32 tensor")
    _need(out.numel() >= rows * width, where, f"out holds {out.numel()} values, the call writes {rows * width}")
    _need(lse.dtype == torch.float32 and lse.is_contiguous() and lse.numel() >= rows, where,
          f"lse must be a contiguous fp32 tensor of at least {rows} values")
    _need(cache.is_contiguous(), where, "cache must be contiguous")
    _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.stride(1) == 1, where,
          "block_table must be a 2-D int32 tensor with contiguous rows")
    B = seq_lens.numel()
    _need(block_table.shape[0] >= B, where, f"block_table has {block_table.shape[0]} rows for {B} requests")
    _need(seq_lens.dtype == torch.int32 and seq_lens.is_contiguous(), where, "seq_lens must be contiguous int32")
    if workspace is not None:
        _need(workspace.is_contiguous(), where, "workspace must be contiguous")


def _write_args(where, latent, k_pe, slot_mapping, cache, status, width):
    """Checks shared by the cache writes: rows of `width` latent values."""
    _on_device(where, latent=latent, k_pe=k_pe, slot_mapping=slot_mapping, cache=cache, status=status)
    _need(latent.dtype == torch.bfloat16 and k_pe.dtype == torch.bfloat16, where, "latent and k_pe must be bf16")
    _need(latent.dim() in (1, 2) and k_pe.dim() in (1, 2) and latent.shape[-1] == width and k_pe.shape[-1] == 64,
          where, f"latent must be [T, {width}] and k_pe [T, 64]")
    _need(latent.stride(-1) == 1 and k_pe.stride(-1) == 1, where, "latent and k_pe rows must be contiguous")
    _need(slot_mapping.dtype == torch.int64 and slot_mapping.is_contiguous(), where,
          "slot_mapping must be contiguous int64")
    T = slot_mapping.numel()
    rows = lambda t: t.shape[0] if t.dim() == 2 else 1
    _need(rows(latent) >= T and rows(k_pe) >= T, where, f"latent / k_pe have fewer than the {T} rows slot_mapping names")
    _need(cache.is_contiguous(), where, "cache must be contiguous")
    _need(status is None or (status.dtype == torch.int32 and status.numel() >= 1), where,
          "status must be an int32 tensor")


def mla_status_string(status: int) -> str:
    try:
        return load().mla_status_string(status).decode()
    except ImportError:
        return f"status {status}"


def mla_row_bytes(cache_kind: int) -> int:
    return load().mla_row_bytes(cache_kind)


def mla_num_sms() -> int:
    return load().mla_num_sms()


def mla_cache_write(latent: torch.Tensor, k_pe: torch.Tensor, slot_mapping: torch.Tensor, cache: torch.Tensor,
                    cache_kind: int = MLA_CACHE_BF16_576, stream=None, status: torch.Tensor = None) -> None:
    """latent [T,512] bf16, k_pe [T,64] bf16 (row-strided views allowed),
    slot_mapping [T] int64 (-1 = skip), cache [num_slots, row_bytes] (any dtype
    viewable as bytes). Scatters rows in place; slots >= num_slots are skipped
    and, when `status` (a device int32 tensor) is given, OR bit 2 into its
    first element."""
    _write_args("mla_cache_write", latent, k_pe, slot_mapping, cache, status, 512)
    T = slot_mapping.numel()
    nbytes = cache.numel() * cache.element_size()
    rb = mla_row_bytes(cache_kind)
    _need(rb > 0, "mla_cache_write", f"unknown cache kind {cache_kind}")
    _check(load().mla_cache_write(latent.data_ptr(), latent.stride(0) if latent.dim() == 2 else 512,
                                  k_pe.data_ptr(), k_pe.stride(0) if k_pe.dim() == 2 else 64,
                                  slot_mapping.data_ptr(), T, cache.data_ptr(), nbytes // rb, cache_kind,
                                  status.data_ptr() if status is not None else None,
                                  _stream(stream)), "mla_cache_write")


def mla_decode_varlen(q_lat, q_pe, cache, cache_kind, page_size, block_table, seq_lens, cu_q_lens, max_q_len,
                      scale, out, lse, workspace, num_ctas: int = 0, stream=None) -> None:
    """Decode with per-request verify lengths (include/mla.h): q_lat [total_q, Hq, 512],
    cu_q_lens int32 [B+1] on the device."""
    where = "mla_decode_varlen"
    _need(isinstance(q_lat, torch.Tensor) and q_lat.dim() == 3, where, "q_lat must be [total_q, Hq, 512]")
    total_q, Hq = q_lat.shape[0], q_lat.shape[1]
    _need(q_lat.shape == (total_q, Hq, 512) and tuple(q_pe.shape) == (total_q, Hq, 64), where,
          "q_lat must be [total_q, Hq, 512] and q_pe [total_q, Hq, 64]")
    _decode_args(where, q_lat, q_pe, cache, block_table, seq_lens, out, lse, workspace, total_q * Hq, 512)
    _on_device(where, q_lat=q_lat, cu_q_lens=cu_q_lens)
    B = seq_lens.numel()
    _need(cu_q_lens.dtype == torch.int32 and cu_q_lens.is_contiguous() and cu_q_lens.numel() == B + 1, where,
          f"cu_q_lens must be contiguous int32 with {B + 1} entries")
    rb = mla_row_bytes(cache_kind)
    _need(rb > 0, where, f"unknown cache kind {cache_kind}")
    odt = MLA_OUT_F32 if out.dtype == torch.float32 else MLA_OUT_BF16
    st = load().mla_decode_varlen(q_lat.data_ptr(), q_pe.data_ptr(), total_q, cache.data_ptr(), int(cache_kind),
                                  _nbytes(cache) // rb, int(page_size), block_table.data_ptr(),
                                  _table_stride(block_table), seq_lens.data_ptr(), cu_q_lens.data_ptr(), B,
                                  int(max_q_len), Hq, float(scale), out.data_ptr(), odt, lse.data_ptr(),
                                  workspace.data_ptr(), _nbytes(workspace), int(num_ctas), _stream(stream))
    _check(st, "mla_decode_varlen")


def mla_gather_upconvert(cache: torch.Tensor, page_size: int, block_table: torch.Tensor, cu_seq_lens: torch.Tensor,
                         dst: torch.Tensor, num_rows: int = None, stream=None) -> None:
    """Context gather of an fp8_ds_mla pool into bf16 rows (include/mla.h)."""
    where = "mla_gather_upconvert"
    _on_device(where, cache=cache, block_table=block_table, cu_seq_lens=cu_seq_lens, dst=dst)
    _need(cache.dtype == torch.uint8 and cache.dim() == 2 and cache.shape[1] == 656 and cache.is_contiguous(), where,
          "cache must be a contiguous uint8 [num_slots, 656] tensor")
    _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.stride(1) == 1, where,
          "block_table must be a 2-D int32 tensor with contiguous rows")
    _need(cu_seq_lens.dtype == torch.int32 and cu_seq_lens.is_contiguous() and cu_seq_lens.numel() >= 1, where,
          "cu_seq_lens must be contiguous int32 with B + 1 entries")
    _need(block_table.shape[0] >= cu_seq_lens.numel() - 1, where, "block_table has fewer rows than requests")
    _need(dst.dtype == torch.bfloat16 and dst.dim() == 2 and dst.stride(1) == 1 and dst.shape[1] >= 576, where,
          "dst must be a bf16 [rows, >= 576] tensor with contiguous rows")
    rows = dst.shape[0] if num_rows is None else int(num_rows)
    _need(0 <= rows <= dst.shape[0], where, f"num_rows {rows} outside [0, {dst.shape[0]}]")
    st = load().mla_gather_upconvert(cache.data_ptr(), cache.shape[0], int(page_size), block_table.data_ptr(),
                                     _table_stride(block_table), cu_seq_lens.data_ptr(), cu_seq_lens.shape[0] - 1, rows,
                                     dst.data_ptr(), dst.stride(0), _stream(stream))
    _check(st, "mla_gather_upconvert")


def mla_cache_write_latent(latent, k_pe, slot_mapping, cache, lat_dim, stream=None, status=None) -> None:
    """bf16 rows [latent lat_dim | rope 64] (include/mla.h): latent
    [T, lat_dim] bf16, k_pe [T, 64] bf16, slot_mapping [T] int64, cache
    [num_slots, 2 (lat_dim + 64)] bytes."""
    _write_args("mla_cache_write_latent", latent, k_pe, slot_mapping, cache, status, int(lat_dim))
    T = slot_mapping.numel()
    row_bytes = 2 * (lat_dim + 64)
    nbytes = cache.numel() * cache.element_size()
    _check(load().mla_cache_write_latent(latent.data_ptr(), latent.stride(0), k_pe.data_ptr(), k_pe.stride(0),
                                         slot_mapping.data_ptr(), T, cache.data_ptr(), nbytes // row_bytes,
                                         int(lat_dim), status.data_ptr() if status is not None else None,
                                         _stream(stream)), "mla_cache_write_latent")


def mla_decode_latent_workspace_bytes(B: int, q_len: int, Hq: int, lat_dim: int, num_ctas: int = 0) -> int:
    n = load().mla_decode_latent_workspace_bytes(B, q_len, Hq, lat_dim, num_ctas)
    if n == 0:
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_decode_latent_workspace_bytes")
    return n


def mla_decode_latent(q_lat, q_pe, cache, lat_dim, page_size, block_table, seq_lens, q_len, scale, out, lse,
                      workspace, num_ctas: int = 0, stream=None) -> None:
    """Decode over bf16 rows of latent width lat_dim (include/mla.h):
    q_lat [B*q_len, Hq, lat_dim], out [B*q_len, Hq, lat_dim]."""
    B = seq_lens.numel()
    Hq = q_lat.shape[-2]
    where = "mla_decode_latent"
    _need(q_lat.shape[-1] == lat_dim and q_pe.shape[-1] == 64 and out.shape[-1] == lat_dim, where,
          f"q_lat and out must end in {lat_dim} values, q_pe in 64")
    _decode_args(where, q_lat, q_pe, cache, block_table, seq_lens, out, lse, workspace, B * int(q_len) * Hq,
                 int(lat_dim))
    out_dtype = MLA_OUT_F32 if out.dtype == torch.float32 else MLA_OUT_BF16
    row_bytes = 2 * (lat_dim + 64)
    nbytes = cache.numel() * cache.element_size()
    _check(load().mla_decode_latent(q_lat.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), int(lat_dim),
                                    nbytes // row_bytes, int(page_size), block_table.data_ptr(),
                                    _table_stride(block_table), seq_lens.data_ptr(), B, int(q_len), Hq, float(scale),
                                    out.data_ptr(), out_dtype, lse.data_ptr(), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), int(num_ctas), _stream(stream)),
           "mla_decode_latent")


def mla_decode_workspace_bytes(B: int, q_len: int, Hq: int, num_ctas: int = 0) -> int:
    n = load().mla_decode_workspace_bytes(B, q_len, Hq, num_ctas)
    if n == 0:
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_decode_workspace_bytes")
    return n


def mla_decode(q_lat, q_pe, cache, cache_kind, page_size, block_table, seq_lens, q_len, scale, out, lse,
               workspace, num_ctas: int = 0, stream=None) -> None:
    """Raw entry point: every buffer is caller-allocated (see include/mla.h)."""
    B = seq_lens.numel()
    Hq = q_lat.shape[-2]
    _decode_args("mla_decode", q_lat, q_pe, cache, block_table, seq_lens, out, lse, workspace, B * int(q_len) * Hq,
                 512)
    out_dtype = MLA_OUT_F32 if out.dtype == torch.float32 else MLA_OUT_BF16
    nbytes = cache.numel() * cache.element_size()
    rb = mla_row_bytes(cache_kind)
    _need(rb > 0, "mla_decode", f"unknown cache kind {cache_kind}")
    _check(load().mla_decode(q_lat.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), cache_kind, nbytes // rb,
                             page_size, block_table.data_ptr(), _table_stride(block_table), seq_lens.data_ptr(), B, q_len,
                             Hq, float(scale), out.data_ptr(), out_dtype, lse.data_ptr(), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), num_ctas, _stream(stream)),
           "mla_decode")


def mla_decode_static_scratch(q_lat, q_pe, cache, cache_kind, page_size, block_table, seq_lens, q_len, scale, out,
                              lse, num_ctas: int = 0, stream=None) -> None:
    """mla_decode with the library's static device scratch as its workspace
    (see include/mla.h: at most MLA_STATIC_SCRATCH_BYTES; calls sharing a
    device must be ordered on one stream)."""
    B = seq_lens.numel()
    Hq = q_lat.shape[-2]
    _decode_args("mla_decode_static_scratch", q_lat, q_pe, cache, block_table, seq_lens, out, lse, None,
                 B * int(q_len) * Hq, 512)
    out_dtype = MLA_OUT_F32 if out.dtype == torch.float32 else MLA_OUT_BF16
    nbytes = cache.numel() * cache.element_size()
    rb = mla_row_bytes(cache_kind)
    _need(rb > 0, "mla_decode_static_scratch", f"unknown cache kind {cache_kind}")
    _check(load().mla_decode_static_scratch(q_lat.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), cache_kind,
                                            nbytes // rb, page_size, block_table.data_ptr(), _table_stride(block_table),
                                            seq_lens.data_ptr(), B, q_len, Hq, float(scale), out.data_ptr(),
                                            out_dtype, lse.data_ptr(), num_ctas, _stream(stream)),
           "mla_decode_static_scratch")


def static_scratch_status_words(n: int = 12, stream=None) -> list:
    """The status words the last mla_decode_static_scratch call on the
    current device left in the static scratch (mla_static_scratch_status):
    word 0 status bits, words 1..11 where a wait gave up (as
    device_status_words for a caller workspace)."""
    dst = torch.zeros(n, dtype=torch.int32, device=torch.cuda.current_device())
    _check(load().mla_static_scratch_status(dst.data_ptr(), n, _stream(stream)), "mla_static_scratch_status")
    return [int(v) for v in dst.tolist()]


def mla_merge_lse(part_out: torch.Tensor, part_lse: torch.Tensor, out: torch.Tensor, lse=None, stream=None) -> None:
    """part_out [S,N,512] fp32, part_lse [S,N] fp32 -> out [N,512] (bf16/fp32), lse [N]."""
    where = "mla_merge_lse"
    _on_device(where, part_out=part_out, part_lse=part_lse, out=out, lse=lse)
    _need(part_lse.dim() == 2, where, "part_lse must be [S, N]")
    S, N = part_lse.shape
    _need(part_out.dtype == torch.float32 and part_lse.dtype == torch.float32, where, "partials must be fp32")
    _need(part_out.is_contiguous() and part_lse.is_contiguous() and part_out.numel() == S * N * 512, where,
          f"part_out must be a contiguous [{S}, {N}, 512] tensor")
    _need(out.dtype in (torch.bfloat16, torch.float32) and out.is_contiguous() and out.numel() >= N * 512, where,
          f"out must be a contiguous bf16 or fp32 tensor of at least {N} x 512 values")
    _need(lse is None or (lse.dtype == torch.float32 and lse.is_contiguous() and lse.numel() >= N), where,
          f"lse must be a contiguous fp32 tensor of at least {N} values")
    out_dtype = MLA_OUT_F32 if out.dtype == torch.float32 else MLA_OUT_BF16
    _check(load().mla_merge_lse(part_out.data_ptr(), part_lse.data_ptr(), S, N, out.data_ptr(), out_dtype,
                                lse.data_ptr() if lse is not None else None, _stream(stream)), "mla_merge_lse")


def _refuse(where, detail) -> None:
    raise MlaError(MLA_ERR_INVALID_ARG, where, detail)


def _row_bytes(where, cache_kind, lat_dim) -> int:
    """Bytes of a cached row; bf16 rows may have another latent width."""
    if cache_kind == MLA_CACHE_BF16_576:
        if lat_dim <= 0:
            _refuse(where, f"lat_dim {lat_dim}")
        return 2 * (lat_dim + 64)
    rb = mla_row_bytes(cache_kind)
    if rb <= 0:
        _refuse(where, f"unknown cache kind {cache_kind}")
    if lat_dim != 512:
        _refuse(where, "rows of this cache kind have lat_dim 512")
    return rb


def _current_device() -> int:
    return torch.cuda.current_device()


def _here(where, names, tensors) -> None:
    """Every tensor (but the last, which need not be given) is a CUDA tensor on
    the current device, where the library launches. A call of a few microseconds
    is mostly its checks, so the common case is a comparison of device numbers."""
    first = tensors[0]
    if _is_cuda(first):
        dev = _current_device()
        try:
            for t in tensors if tensors[-1] is not None else tensors[:-1]:
                if t.get_device() != dev:
                    break
            else:
                return
        except AttributeError:  # not a tensor
            pass
    for name, t in zip(names, tensors[:-1]):
        if not _is_cuda(t):
            _refuse(where, f"{name} must be a CUDA tensor")
    _on_device(where, **dict(zip(names, tensors)))
    _refuse(where, f"the arguments are on {first.device}, the current device is cuda:{_current_device()}")


def _rows_apart(shape, strides) -> bool:
    """Whether a tensor is 2-D with contiguous rows that do not share elements."""
    if len(shape) != 2:
        return False
    rows, cols = shape
    s0, s1 = strides
    return (s1 == 1 or cols <= 1) and (s0 >= cols or rows <= 1)


def _status_ptr(where, status):
    if status is None:
        return None
    if status.dtype is not torch.int32 or status.numel() < 1:
        _refuse(where, "status must be an int32 tensor")
    return status.data_ptr()


def _one_row_stride(block_table, stride, cols) -> int:
    """_table_stride of a table of one row, cut to what lies in memory."""
    if stride <= cols:
        return cols
    return max(cols, min(stride, block_table.untyped_storage().nbytes() // 4 - block_table.storage_offset()))


def _table_args(where, block_table, seq_lens, cache, max_len, page_size):
    """Checks of a paged batch shared by the calls that keep the cache: the number
    of requests and the table's row stride."""
    if not cache.is_contiguous():
        _refuse(where, "cache must be contiguous")
    shape, strides, i32 = block_table.shape, block_table.stride(), torch.int32
    if block_table.dtype is not i32 or len(shape) != 2 or strides[1] != 1:
        _refuse(where, "block_table must be a 2-D int32 tensor with contiguous rows")
    if seq_lens.dtype is not i32 or not seq_lens.is_contiguous():
        _refuse(where, "seq_lens must be contiguous int32")
    B = seq_lens.numel()
    rows, cols = shape
    if rows < B:
        _refuse(where, f"block_table has {rows} rows for {B} requests")
    stride = strides[0]
    if max_len == 0:
        stride = max(stride, 1)  # nothing is read
    elif rows == 1:
        stride = _one_row_stride(block_table, stride, cols)
    elif stride < cols and rows > 0:
        _refuse(where, "block_table's rows overlap")
    elif stride > cols and B > 0 and page_size > 0:
        # columns of a wider table: a row reaches to the next one, as far as max_len
        # goes, and the last must lie in memory as well
        last = (B - 1) * stride + min(stride, -(-max_len // page_size))
        if last > block_table.untyped_storage().nbytes() // 4 - block_table.storage_offset():
            _refuse(where, f"block_table's last row ends before the pages of {max_len} tokens")
    return B, stride


_PREFILL_NAMES = ("q", "k_nope", "k_pe", "v", "cu_q_lens", "cu_k_lens", "out", "lse", "status")


def mla_prefill(q, k_nope, k_pe, v, cu_q_lens, cu_k_lens, max_q_len, scale, out, lse, causal: bool = True, status=None,
                stream=None) -> None:
    """Attention over whole packed prompts (include/mla.h): q [total_q, Hq, 192],
    k_nope and v [total_k, Hkv, 128], k_pe [total_k, 64], all bf16 with
    contiguous last dimensions (strided views allowed), cu_q_lens and cu_k_lens
    int32 [B + 1] on the device, out bf16 [total_q, Hq, 128], lse fp32
    [total_q, Hq]. `status` (a device int32 tensor) collects status bits."""
    where = "mla_prefill"
    _here(where, _PREFILL_NAMES, (q, k_nope, k_pe, v, cu_q_lens, cu_k_lens, out, lse, status))
    bf16 = torch.bfloat16
    q_shape, kv_shape = q.shape, k_nope.shape
    if len(q_shape) != 3 or q_shape[2] != 192:
        _refuse(where, "q must be [total_q, Hq, 192]")
    if len(kv_shape) != 3 or kv_shape[2] != 128:
        _refuse(where, "k_nope must be [total_k, Hkv, 128]")
    total_q, Hq, _ = q_shape
    total_k, Hkv, _ = kv_shape
    if v.shape != kv_shape:
        _refuse(where, "v must have k_nope's shape")
    if k_pe.shape != (total_k, 64):
        _refuse(where, f"k_pe must be [{total_k}, 64]")
    sq, sk, sp, sv = q.stride(), k_nope.stride(), k_pe.stride(), v.stride()
    if (q.dtype is not bf16 or k_nope.dtype is not bf16 or k_pe.dtype is not bf16 or v.dtype is not bf16 or
            sq[2] != 1 or sk[2] != 1 or sp[1] != 1 or sv[2] != 1):
        _refuse(where, "q must be bf16 with a contiguous last dimension, and so must k_nope, k_pe and v")
    if out.dtype is not bf16 or out.shape != (total_q, Hq, 128) or not out.is_contiguous():
        _refuse(where, f"out must be a contiguous bf16 [{total_q}, {Hq}, 128] tensor")
    if lse.dtype is not torch.float32 or lse.shape != (total_q, Hq) or not lse.is_contiguous():
        _refuse(where, f"lse must be a contiguous fp32 [{total_q}, {Hq}] tensor")
    B = cu_q_lens.numel() - 1
    i32 = torch.int32
    if cu_q_lens.dtype is not i32 or not cu_q_lens.is_contiguous() or B < 0:
        _refuse(where, "cu_q_lens must be contiguous int32 with B + 1 entries")
    if cu_k_lens.dtype is not i32 or not cu_k_lens.is_contiguous() or cu_k_lens.numel() != B + 1:
        _refuse(where, "cu_k_lens must be contiguous int32 with as many entries as cu_q_lens")
    st = _status_ptr(where, status)
    # (the stride of a dimension of one entry says nothing)
    one_q, one_k, one_h, one_g = total_q <= 1, total_k <= 1, Hq <= 1, Hkv <= 1
    _check(load().mla_prefill(
        q.data_ptr(), 192 if one_q else sq[0], 192 if one_h else sq[1],
        k_nope.data_ptr(), 128 if one_k else sk[0], 128 if one_g else sk[1], k_pe.data_ptr(), 64 if one_k else sp[0],
        v.data_ptr(), 128 if one_k else sv[0], 128 if one_g else sv[1], cu_q_lens.data_ptr(), cu_k_lens.data_ptr(), B,
        total_q, total_k, int(max_q_len), Hq, Hkv, 1 if causal else 0, float(scale), out.data_ptr(), lse.data_ptr(), st,
        _stream(stream)), where)


_WEIGHTS_NAMES = ("q_lat", "q_pe", "lse", "cache", "block_table", "seq_lens", "weights", "status")


def mla_attn_weights(q_lat, q_pe, lse, cache, cache_kind, page_size, block_table, seq_lens, q_len, scale, weights,
                     decay: float = 0.0, lat_dim: int = 512, num_ctas: int = 0, status=None, stream=None) -> None:
    """weights[b][j] = decay * weights[b][j] + the attention that token j of
    request b received from the step's queries (include/mla.h): q_lat
    [B*q_len, Hq, lat_dim] and q_pe [B*q_len, Hq, 64] bf16 as in mla_decode,
    lse [B*q_len, Hq] fp32 from it, weights fp32 [>= B, max_len] with
    contiguous rows. `status` (a device int32 tensor) collects status bits."""
    where = "mla_attn_weights"
    _here(where, _WEIGHTS_NAMES, (q_lat, q_pe, lse, cache, block_table, seq_lens, weights, status))
    w_shape, w_strides = weights.shape, weights.stride()
    max_len = w_shape[-1] if w_shape else 0
    B, bt_stride = _table_args(where, block_table, seq_lens, cache, max_len, int(page_size))
    q_shape = q_lat.shape
    Hq = q_shape[-2] if len(q_shape) >= 2 else 0
    rows = B * int(q_len) * Hq
    bf16, f32 = torch.bfloat16, torch.float32
    if q_lat.dtype is not bf16 or q_pe.dtype is not bf16:
        _refuse(where, "q_lat and q_pe must be bf16")
    if not q_lat.is_contiguous() or not q_pe.is_contiguous():
        _refuse(where, "q_lat and q_pe must be contiguous")
    if q_lat.numel() != rows * lat_dim or q_pe.numel() != rows * 64:
        _refuse(where, f"q_lat / q_pe hold {q_lat.numel()} / {q_pe.numel()} values, {rows} rows of {lat_dim} / 64 expected")
    if lse.dtype is not f32 or not lse.is_contiguous() or lse.numel() != rows:
        _refuse(where, f"lse must be a contiguous fp32 tensor of {rows} values")
    if weights.dtype is not f32 or not _rows_apart(w_shape, w_strides) or w_shape[0] < B:
        _refuse(where, f"weights must be a fp32 [>= {B}, max_len] tensor with contiguous rows")
    st = _status_ptr(where, status)
    rb = _row_bytes(where, cache_kind, lat_dim)
    _check(load().mla_attn_weights(
        q_lat.data_ptr(), q_pe.data_ptr(), lse.data_ptr(), cache.data_ptr(), int(cache_kind), int(lat_dim),
        cache.nbytes // rb, int(page_size), block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), B,
        int(q_len), Hq, float(scale), float(decay),
        weights.data_ptr(), max(w_strides[0], max_len), max_len, st, int(num_ctas), _stream(stream)), where)


_EVICT_NAMES = ("cache", "block_table", "seq_lens", "weights", "positions", "budgets", "new_seq_lens", "new_weights",
                "new_positions", "moves", "status")


def mla_cache_evict(cache, cache_kind, page_size, block_table, seq_lens, weights, positions, budgets, n_sink,
                    n_recent, new_seq_lens, new_weights, new_positions, moves, lat_dim: int = 512, status=None,
                    stream=None) -> None:
    """Keep each request's budgets[b] best-scored tokens and close the gaps in
    its pages, in place (include/mla.h): weights fp32 and positions int32
    [>= B, max_len] with the same row stride, budgets int32 [B]; new_seq_lens
    int32 [B], new_weights and new_positions shaped as the inputs (or the
    inputs themselves), moves int32 [>= B, >= max_len + 2]."""
    where = "mla_cache_evict"
    _here(where, _EVICT_NAMES, (cache, block_table, seq_lens, weights, positions, budgets, new_seq_lens, new_weights,
                                new_positions, moves, status))
    shape, strides, f32, i32 = weights.shape, weights.stride(), torch.float32, torch.int32
    max_len = shape[-1] if shape else 0
    B, bt_stride = _table_args(where, block_table, seq_lens, cache, max_len, int(page_size))
    if not _rows_apart(shape, strides) or shape[0] < B:
        _refuse(where, f"weights must be [>= {B}, max_len] with contiguous rows")
    if (weights.dtype is not f32 or positions.dtype is not i32 or new_weights.dtype is not f32 or
            new_positions.dtype is not i32):
        _refuse(where, "weights and new_weights must be fp32, positions and new_positions int32")
    # (one row: its stride says nothing, but its values still have to follow each other)
    one = shape[0] <= 1
    for name, t in (("positions", positions), ("new_weights", new_weights), ("new_positions", new_positions)):
        if t.shape != shape or (not _rows_apart(shape, t.stride()) if one else t.stride() != strides):
            _refuse(where, f"{name} must be a tensor of weights' shape and strides")
    if budgets.dtype is not i32 or not budgets.is_contiguous() or budgets.numel() < B:
        _refuse(where, f"budgets must be contiguous int32 of at least {B} values")
    if new_seq_lens.dtype is not i32 or not new_seq_lens.is_contiguous() or new_seq_lens.numel() < B:
        _refuse(where, f"new_seq_lens must be contiguous int32 of at least {B} values")
    m_shape, m_strides = moves.shape, moves.stride()
    if moves.dtype is not i32 or not _rows_apart(m_shape, m_strides) or m_shape[0] < B or m_shape[1] < max_len + 2:
        _refuse(where, f"moves must be an int32 [>= {B}, >= {max_len + 2}] tensor")
    st = _status_ptr(where, status)
    rb = _row_bytes(where, cache_kind, lat_dim)
    _check(load().mla_cache_evict(
        cache.data_ptr(), int(rb), cache.nbytes // rb, int(page_size), block_table.data_ptr(), bt_stride,
        seq_lens.data_ptr(), weights.data_ptr(), positions.data_ptr(), max(strides[0], max_len), max_len,
        budgets.data_ptr(), B, int(n_sink), int(n_recent), new_seq_lens.data_ptr(), new_weights.data_ptr(),
        new_positions.data_ptr(), moves.data_ptr(), max(m_strides[0], m_shape[1]), st, _stream(stream)), where)


def decode(q_lat, q_pe, cache, cache_kind, page_size, block_table, seq_lens, q_len, scale,
           out_dtype=torch.bfloat16, num_ctas: int = 0, workspace=None, stream=None):
    """Allocate out/lse (and the workspace unless given) and run mla_decode.
    Returns (out [B*q_len, Hq, 512], lse [B*q_len, Hq], workspace)."""
    B = seq_lens.numel()
    Hq = q_lat.shape[-2]
    dev = q_lat.device
    out = torch.empty((B * q_len, Hq, 512), dtype=out_dtype, device=dev)
    lse = torch.empty((B * q_len, Hq), dtype=torch.float32, device=dev)
    need = mla_decode_workspace_bytes(B, q_len, Hq, num_ctas)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    mla_decode(q_lat, q_pe, cache, cache_kind, page_size, block_table, seq_lens, q_len, scale, out, lse, workspace,
               num_ctas, stream)
    return out, lse, workspace


def device_status_words(workspace: torch.Tensor, n: int = 12) -> list:
    """The workspace status header of the last mla_decode that used it:
    word 0 status bits, words 1..3 the first failing CTA's wait site, tile and
    index, words 4..11 where each of its roles gave up ((site << 24) | tile)."""
    return [int(v) for v in workspace[:4 * n].view(torch.int32).tolist()]


def test_hold_next_decode() -> None:
    """Test support: make the next mla_decode's PV issuers time out (see
    include/mla.h)."""
    load().mla_test_hold_next_decode()


def test_slow_pv_next_decode() -> None:
    """Test support: make one PV issuer of the next mla_decode lag the
    softmax warps by up to two tiles; its results are unchanged (see
    include/mla.h)."""
    load().mla_test_slow_pv_next_decode()


def test_limit_next_evict(ctas: int) -> None:
    """Test support: at most `ctas` CTAs share a request's tokens in the next
    mla_cache_evict; its results are unchanged (see include/mla.h)."""
    load().mla_test_limit_next_evict(int(ctas))


def device_status(workspace: torch.Tensor) -> int:
    """Device-side status word of the last mla_decode that used `workspace`
    (0 = ok; bit 1 = a bounded wait gave up; bit 2 = a block id outside the
    pool or a page index past the table row; bit 4 = an fp8 value past the
    f16 range of the fp8 path up to 64 rows)."""
    return int(workspace[:4].view(torch.int32).item())
