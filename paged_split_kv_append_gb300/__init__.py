"""Python binding of libnbx: paged KV append and split-KV decode attention on GB300.

Argument marshalling only: every function takes torch tensors, checks their dtypes,
shapes and devices, and calls the C entry point of the same name in libnbx.so with
raw device pointers and the current CUDA stream. All computation runs in the
library's CUDA kernels; there is no other code path. If libnbx.so is missing the
first call raises ``NbxLibraryMissing`` (build it with ``build()``).

The C ABI is declared in ``include/nbx.h``.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

from . import _build

__all__ = [
    "NBX_F32", "NBX_BF16", "NBX_E4M3", "NbxError", "NbxLibraryMissing", "build", "lib", "library_path",
    "nbx_paged_kv_append", "nbx_paged_decode_workspace_bytes", "nbx_paged_decode_attn",
    "nbx_paged_decode_merge", "nbx_set_decode_grid_limit", "nbx_set_decode_wait_test", "nbx_status_string",
    "nbx_paged_decode_bounds", "nbx_paged_decode_attn_fixed_shift", "nbx_decode_fixed_shift_gate",
    "nbx_paged_kv_append_block_scaled", "nbx_paged_decode_attn_block_scaled", "nbx_paged_decode_attn_modified",
    "nbx_paged_decode_modified_workspace_bytes", "nbx_paged_decode_modified_partial_kernel",
    "nbx_paged_kv_copy_pages", "nbx_paged_kv_fork",
    "nbx_paged_kv_fork_workspace_bytes", "nbx_paged_kv_compact", "nbx_paged_kv_compact_workspace_bytes",
    "dtype_code",
    "DEV_BAD_SLOT", "DEV_BAD_PAGE", "DEV_BAD_LEN", "DEV_TIMEOUT", "DEV_BAD_SCALE", "DEV_BAD_ROW", "DEV_NO_PAGE",
]

NBX_F32, NBX_BF16, NBX_E4M3 = 0, 1, 2
DEV_BAD_SLOT, DEV_BAD_PAGE, DEV_BAD_LEN, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEV_BAD_SCALE, DEV_BAD_ROW, DEV_NO_PAGE = 0x10, 0x20, 0x40
PARTIAL_SIMT, PARTIAL_TCGEN05, PARTIAL_TCGEN05_FP8, PARTIAL_WARP = 0, 1, 2, 3

_lib = None
_lock = threading.Lock()


class NbxError(RuntimeError):
    def __init__(self, func: str, status: int):
        super().__init__(f"{func}: {nbx_status_string(status)} (status {status})")
        self.status = status


class NbxLibraryMissing(RuntimeError):
    pass


def library_path() -> str:
    return _build.LIB


def build(force: bool = False) -> str:
    """Compile libnbx.so for sm_103a in-tree (nvcc) and return its path."""
    return _build.build(force=force)


def _declare(l):
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    l.nbx_paged_kv_append.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, i32, i32, i32, vp, f32, f32, vp, vp]
    l.nbx_paged_kv_append.restype = i32
    l.nbx_paged_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    l.nbx_paged_decode_workspace_bytes.restype = sz
    l.nbx_paged_decode_workspace_bytes_for.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32]
    l.nbx_paged_decode_workspace_bytes_for.restype = sz
    l.nbx_paged_decode_attn.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp, i32,
                                        f32, f32, f32, vp, vp, sz, vp, vp]
    l.nbx_paged_decode_attn.restype = i32
    l.nbx_paged_decode_step.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, i32,
                                        vp, i32, f32, f32, f32, vp, vp, sz, vp, vp]
    l.nbx_paged_decode_step.restype = i32
    l.nbx_decode_attn_contiguous.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, i32, i32, i32, vp, i32, f32, f32, f32,
                                             vp, vp, sz, vp, vp]
    l.nbx_decode_attn_contiguous.restype = i32
    l.nbx_paged_decode_merge.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
    l.nbx_paged_decode_merge.restype = i32
    l.nbx_paged_decode_partial_kernel.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
    l.nbx_paged_decode_partial_kernel.restype = i32
    l.nbx_set_decode_grid_limit.argtypes = [i32]
    l.nbx_set_decode_grid_limit.restype = None
    l.nbx_set_decode_wait_test.argtypes = [ctypes.c_ulonglong, ctypes.c_ulonglong]
    l.nbx_set_decode_wait_test.restype = None
    l.nbx_paged_decode_bounds.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp, i32,
                                          f32, f32, vp, vp, vp, vp]
    l.nbx_paged_decode_bounds.restype = i32
    l.nbx_paged_decode_attn_fixed_shift.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, i32, i32, i32, i32, vp, i32,
                                                    vp, i32, f32, f32, f32, vp, vp, sz, vp, vp, vp, vp]
    l.nbx_paged_decode_attn_fixed_shift.restype = i32
    l.nbx_decode_fixed_shift_gate.argtypes = [i32, ctypes.c_double, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    l.nbx_decode_fixed_shift_gate.restype = i32
    l.nbx_paged_kv_append_block_scaled.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, i32, i32, i32, vp, i32,
                                                   i32, vp, vp, vp, vp]
    l.nbx_paged_kv_append_block_scaled.restype = i32
    l.nbx_paged_decode_modified_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    l.nbx_paged_decode_modified_workspace_bytes.restype = sz
    l.nbx_paged_decode_modified_partial_kernel.argtypes = [i32] * 9
    l.nbx_paged_decode_modified_partial_kernel.restype = i32
    l.nbx_paged_decode_attn_block_scaled.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, i32, i32, i32, i32,
                                                     vp, i32, vp, i32, f32, f32, vp, vp, vp, vp, i32, vp, sz, vp, vp]
    l.nbx_paged_decode_attn_block_scaled.restype = i32
    l.nbx_paged_decode_attn_modified.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp,
                                                 i32, f32, f32, f32, f32, vp, vp, vp, vp, i32, vp, sz, vp, vp]
    l.nbx_paged_decode_attn_modified.restype = i32
    l.nbx_paged_kv_copy_pages.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp]
    l.nbx_paged_kv_copy_pages.restype = i32
    l.nbx_paged_kv_fork_workspace_bytes.argtypes = [i32, i32, i32, i32]
    l.nbx_paged_kv_fork_workspace_bytes.restype = sz
    l.nbx_paged_kv_fork.argtypes = [vp, i32, vp, i32, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp,
                                    vp, sz, vp, vp]
    l.nbx_paged_kv_fork.restype = i32
    l.nbx_paged_kv_compact_workspace_bytes.argtypes = [i32]
    l.nbx_paged_kv_compact_workspace_bytes.restype = sz
    l.nbx_paged_kv_compact.argtypes = [vp, vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, vp, i32, vp,
                                       vp, sz, vp, vp]
    l.nbx_paged_kv_compact.restype = i32
    l.nbx_call.argtypes = [i32, ctypes.c_char_p]
    l.nbx_call.restype = i32
    l.nbx_status_string.argtypes = [i32]
    l.nbx_status_string.restype = ctypes.c_char_p
    l.nbx_abi_version.argtypes = []
    l.nbx_abi_version.restype = i32


def lib() -> ctypes.CDLL:
    """The loaded libnbx.so (loaded once, on first use)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise NbxLibraryMissing(f"libnbx.so not found at {path}: run paged_split_kv_append_gb300.build()")
            l = ctypes.CDLL(path)
            _declare(l)
            _lib = l
    return _lib


_DTYPES = {torch.float32: NBX_F32, torch.bfloat16: NBX_BF16, torch.float8_e4m3fn: NBX_E4M3, torch.uint8: NBX_E4M3}


def dtype_code(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def nbx_status_string(status: int) -> str:
    return lib().nbx_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(func: str, status: int):
    if status != 0:
        raise NbxError(func, status)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _new(shape, dtype, like: torch.Tensor, stream, fill=None) -> torch.Tensor:
    """A tensor on `like`'s device for a call on `stream`, uninitialised or filled. For a stream that is not the
    current one the memory comes from that stream's own (the current one may have work to do on what it has freed),
    the filling is that stream's work, and the allocator learns that the current one may use the tensor too."""
    dev = like.get_device()
    handle = None if stream is None else int(getattr(stream, "cuda_stream", stream))
    if handle is None or handle == _raw_stream(dev):
        t = torch.empty(shape, dtype=dtype, device=like.device)
        return t if fill is None else t.fill_(fill)
    current = torch.cuda.current_stream(dev)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=like.device)):
        t = torch.empty(shape, dtype=dtype, device=like.device)
        if fill is not None:
            t.fill_(fill)
    t.record_stream(current)
    return t


def _cuda_contig(name: str, t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def nbx_paged_kv_append(new_k: torch.Tensor, new_v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                        slot_mapping: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """new_k / new_v [n_tok, h_kv, d] (fp32 or bf16) into the pools [num_pages, h_kv, page_tokens, d]
    (fp32, bf16 or e4m3) at slot_mapping [n_tok] int32; cast on store."""
    for n, t in (("new_k", new_k), ("new_v", new_v), ("k_pool", k_pool), ("v_pool", v_pool),
                 ("slot_mapping", slot_mapping)):
        _cuda_contig(n, t)
    if slot_mapping.dtype != torch.int32:
        raise ValueError("slot_mapping must be int32")
    if new_k.shape != new_v.shape or k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("K and V must have the same shapes and dtypes")
    n_tok, h_kv, d = new_k.shape
    num_pages, h_kv_p, page_tokens, d_p = k_pool.shape
    if (h_kv_p, d_p) != (h_kv, d) or slot_mapping.numel() != n_tok:
        raise ValueError(f"new {list(new_k.shape)} does not fit the pool {list(k_pool.shape)}")
    st = lib().nbx_paged_kv_append(_ptr(new_k), _ptr(new_v), dtype_code(new_k), n_tok, h_kv, d, _ptr(k_pool),
                                   _ptr(v_pool), dtype_code(k_pool), num_pages, page_tokens, _ptr(slot_mapping),
                                   float(k_scale), float(v_scale), _ptr(status), _stream(stream))
    _check("nbx_paged_kv_append", st)


def nbx_paged_decode_workspace_bytes(batch: int, rows: int, h_q: int, h_kv: int, d: int, max_seq_len: int) -> int:
    return int(lib().nbx_paged_decode_workspace_bytes(batch, rows, h_q, h_kv, d, max_seq_len))


def nbx_paged_decode_workspace_bytes_for(q_dtype: int, pool_dtype: int, batch: int, rows: int, h_q: int, h_kv: int,
                                         d: int, max_seq_len: int, page_tokens: int) -> int:
    return int(lib().nbx_paged_decode_workspace_bytes_for(q_dtype, pool_dtype, batch, rows, h_q, h_kv, d,
                                                          max_seq_len, page_tokens))


def nbx_paged_decode_attn(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: torch.Tensor,
                          seq_lens: torch.Tensor, max_seq_len: int, scale: float, k_scale: float = 1.0,
                          v_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """q [batch, rows, h_q, d] (fp32 or bf16), pools [num_pages, h_kv, page_tokens, d], block_table
    [batch, max_pages] int32 (-1 padded), seq_lens [batch] int32 -> out [batch, rows, h_q, d] fp32."""
    for n, t in (("q", q), ("k_pool", k_pool), ("v_pool", v_pool), ("block_table", block_table),
                 ("seq_lens", seq_lens)):
        _cuda_contig(n, t)
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_table and seq_lens must be int32")
    if k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("k_pool and v_pool must match")
    batch, rows, h_q, d = q.shape
    num_pages, h_kv, page_tokens, d_p = k_pool.shape
    if d_p != d or block_table.dim() != 2 or block_table.shape[0] != batch or seq_lens.numel() != batch:
        raise ValueError(f"q {list(q.shape)}, pool {list(k_pool.shape)}, block_table {list(block_table.shape)}, "
                         f"seq_lens {list(seq_lens.shape)} do not fit")
    max_pages = block_table.shape[1]
    if out is None:
        out = _new((batch, rows, h_q, d), torch.float32, q, stream)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_pool), batch, rows, h_q, h_kv, d,
                                                max_seq_len, page_tokens)
    if workspace is None:
        workspace = _new(max(need, 256), torch.uint8, q, stream)
    st = lib().nbx_paged_decode_attn(_ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(k_pool), _ptr(v_pool),
                                     dtype_code(k_pool), num_pages, h_kv, page_tokens, _ptr(block_table), max_pages,
                                     _ptr(seq_lens), int(max_seq_len), float(scale), float(k_scale),
                                     float(v_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                     _ptr(status), _stream(stream))
    _check("nbx_paged_decode_attn", st)
    return out


def nbx_paged_decode_step(q: torch.Tensor, new_k: torch.Tensor, new_v: torch.Tensor, k_pool: torch.Tensor,
                          v_pool: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, max_seq_len: int,
                          scale: float, k_scale: float = 1.0, v_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """One decode step: new_k/new_v [batch, rows, h_kv, d] (fp32 or bf16) are written at positions
    lens[b] .. lens[b] + rows - 1, the rows of q [batch, rows, h_q, d] attend, and lens [batch] int32
    advances by rows, all on the stream. Returns out [batch, rows, h_q, d] fp32."""
    for n, t in (("q", q), ("new_k", new_k), ("new_v", new_v), ("k_pool", k_pool), ("v_pool", v_pool),
                 ("block_table", block_table), ("lens", lens)):
        _cuda_contig(n, t)
    if block_table.dtype != torch.int32 or lens.dtype != torch.int32:
        raise ValueError("block_table and lens must be int32")
    if k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype or new_k.shape != new_v.shape or \
            new_k.dtype != new_v.dtype:
        raise ValueError("k/v tensors must match")
    batch, rows, h_q, d = q.shape
    num_pages, h_kv, page_tokens, d_p = k_pool.shape
    if d_p != d or tuple(new_k.shape) != (batch, rows, h_kv, d) or block_table.dim() != 2 or \
            block_table.shape[0] != batch or lens.numel() != batch:
        raise ValueError(f"q {list(q.shape)}, new_k {list(new_k.shape)}, pool {list(k_pool.shape)}, "
                         f"block_table {list(block_table.shape)}, lens {list(lens.shape)} do not fit")
    if out is None:
        out = _new((batch, rows, h_q, d), torch.float32, q, stream)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_pool), batch, rows, h_q, h_kv, d,
                                                max_seq_len, page_tokens)
    if workspace is None:
        workspace = _new(max(need, 256), torch.uint8, q, stream)
    st = lib().nbx_paged_decode_step(_ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(new_k), _ptr(new_v),
                                     dtype_code(new_k), _ptr(k_pool), _ptr(v_pool), dtype_code(k_pool), num_pages,
                                     h_kv, page_tokens, _ptr(block_table), block_table.shape[1], _ptr(lens),
                                     int(max_seq_len), float(scale), float(k_scale), float(v_scale), _ptr(out),
                                     _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _check("nbx_paged_decode_step", st)
    return out


def nbx_decode_attn_contiguous(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seq_lens: torch.Tensor,
                               max_seq_len: int, scale: float, k_scale: float = 1.0, v_scale: float = 1.0,
                               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                               status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """q [batch, rows, h_q, d], caches [batch, h_kv, capacity, d] (no page table), seq_lens [batch]
    int32 -> out [batch, rows, h_q, d] fp32."""
    for n, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("seq_lens", seq_lens)):
        _cuda_contig(n, t)
    if seq_lens.dtype != torch.int32:
        raise ValueError("seq_lens must be int32")
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must match")
    batch, rows, h_q, d = q.shape
    b_c, h_kv, capacity, d_c = k_cache.shape
    if b_c != batch or d_c != d or seq_lens.numel() != batch:
        raise ValueError(f"q {list(q.shape)}, cache {list(k_cache.shape)}, seq_lens {list(seq_lens.shape)} do not fit")
    if out is None:
        out = _new((batch, rows, h_q, d), torch.float32, q, stream)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_cache), batch, rows, h_q, h_kv, d,
                                                max_seq_len, capacity)
    if workspace is None:
        workspace = _new(max(need, 256), torch.uint8, q, stream)
    st = lib().nbx_decode_attn_contiguous(_ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(k_cache), _ptr(v_cache),
                                          dtype_code(k_cache), h_kv, capacity, _ptr(seq_lens), int(max_seq_len),
                                          float(scale), float(k_scale), float(v_scale), _ptr(out), _ptr(workspace),
                                          workspace.numel(), _ptr(status), _stream(stream))
    _check("nbx_decode_attn_contiguous", st)
    return out


def nbx_paged_decode_merge(acc_part: torch.Tensor, m_part: torch.Tensor, l_part: torch.Tensor,
                           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """acc_part [n_rows, splits, d], m_part / l_part [n_rows, splits] fp32 (m in natural-log units)
    -> out [n_rows, d] fp32."""
    for n, t in (("acc_part", acc_part), ("m_part", m_part), ("l_part", l_part)):
        _cuda_contig(n, t)
        if t.dtype != torch.float32:
            raise ValueError(f"{n} must be fp32")
    n_rows, splits, d = acc_part.shape
    if out is None:
        out = _new((n_rows, d), torch.float32, acc_part, stream)
    st = lib().nbx_paged_decode_merge(_ptr(acc_part), _ptr(m_part), _ptr(l_part), n_rows, splits, d, _ptr(out),
                                      _stream(stream))
    _check("nbx_paged_decode_merge", st)
    return out


def nbx_paged_decode_partial_kernel(q_dtype: int, pool_dtype: int, rows: int, h_q: int, h_kv: int, d: int,
                                    num_pages: int, page_tokens: int) -> int:
    """PARTIAL_SIMT or PARTIAL_TCGEN05: the split-partial kernel a decode with these sizes runs."""
    k = lib().nbx_paged_decode_partial_kernel(q_dtype, pool_dtype, rows, h_q, h_kv, d, num_pages, page_tokens)
    _check("nbx_paged_decode_partial_kernel", k if k < 0 else 0)
    return k


def nbx_set_decode_grid_limit(max_ctas: int) -> None:
    lib().nbx_set_decode_grid_limit(int(max_ctas))


def nbx_set_decode_wait_test(wait_limit_ns: int = 0, producer_delay_ns: int = 0) -> None:
    """Tests of the timeout path only: the SIMT partial kernel's wait bound (0 = the default 2 s) and
    a delay before its producer warps start (0 = none)."""
    lib().nbx_set_decode_wait_test(int(wait_limit_ns), int(producer_delay_ns))


def _decode_shapes(q, k_pool, v_pool, block_table, seq_lens):
    for n, t in (("q", q), ("k_pool", k_pool), ("v_pool", v_pool), ("block_table", block_table),
                 ("seq_lens", seq_lens)):
        _cuda_contig(n, t)
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_table and seq_lens must be int32")
    if k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("k_pool and v_pool must match")
    batch, rows, h_q, d = q.shape
    num_pages, h_kv, page_tokens, d_p = k_pool.shape
    if d_p != d or block_table.dim() != 2 or block_table.shape[0] != batch or seq_lens.numel() != batch:
        raise ValueError(f"q {list(q.shape)}, pool {list(k_pool.shape)}, block_table {list(block_table.shape)}, "
                         f"seq_lens {list(seq_lens.shape)} do not fit")
    return batch, rows, h_q, d, num_pages, h_kv, page_tokens, block_table.shape[1]


def nbx_paged_decode_bounds(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: torch.Tensor,
                            seq_lens: torch.Tensor, max_seq_len: int, k_scale: float = 1.0, v_scale: float = 1.0,
                            status: Optional[torch.Tensor] = None, stream=None):
    """The fixed-shift softmax's score bounds: (q_norm [batch, rows, h_q], kv_max [batch, h_kv, 2]) fp32."""
    batch, rows, h_q, d, num_pages, h_kv, page_tokens, max_pages = _decode_shapes(q, k_pool, v_pool, block_table,
                                                                                  seq_lens)
    q_norm = _new((batch, rows, h_q), torch.float32, q, stream)
    kv_max = _new((batch, h_kv, 2), torch.float32, q, stream)
    st = lib().nbx_paged_decode_bounds(_ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(k_pool), _ptr(v_pool),
                                       dtype_code(k_pool), num_pages, h_kv, page_tokens, _ptr(block_table), max_pages,
                                       _ptr(seq_lens), int(max_seq_len), float(k_scale), float(v_scale), _ptr(q_norm),
                                       _ptr(kv_max), _ptr(status), _stream(stream))
    _check("nbx_paged_decode_bounds", st)
    return q_norm, kv_max


def nbx_paged_decode_attn_fixed_shift(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                      block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                                      scale: float, q_norm: torch.Tensor, kv_max: torch.Tensor, k_scale: float = 1.0,
                                      v_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                                      workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                      stream=None) -> torch.Tensor:
    """nbx_paged_decode_attn with the fixed-shift softmax where the bounds pass the gate."""
    batch, rows, h_q, d, num_pages, h_kv, page_tokens, max_pages = _decode_shapes(q, k_pool, v_pool, block_table,
                                                                                  seq_lens)
    _cuda_contig("q_norm", q_norm)
    _cuda_contig("kv_max", kv_max)
    if q_norm.dtype != torch.float32 or kv_max.dtype != torch.float32 or q_norm.numel() != batch * rows * h_q or \
            kv_max.numel() != batch * h_kv * 2:
        raise ValueError("q_norm [batch, rows, h_q] and kv_max [batch, h_kv, 2] must be fp32")
    if out is None:
        out = _new((batch, rows, h_q, d), torch.float32, q, stream)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_pool), batch, rows, h_q, h_kv, d,
                                                max_seq_len, page_tokens)
    if workspace is None:
        workspace = _new(max(need, 256), torch.uint8, q, stream)
    st = lib().nbx_paged_decode_attn_fixed_shift(_ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(k_pool),
                                                 _ptr(v_pool), dtype_code(k_pool), num_pages, h_kv, page_tokens,
                                                 _ptr(block_table), max_pages, _ptr(seq_lens), int(max_seq_len),
                                                 float(scale), float(k_scale), float(v_scale), _ptr(out),
                                                 _ptr(workspace), workspace.numel(), _ptr(q_norm), _ptr(kv_max),
                                                 _ptr(status), _stream(stream))
    _check("nbx_paged_decode_attn_fixed_shift", st)
    return out


def nbx_decode_fixed_shift_gate(n_keys: int, v_max_bound: float = 256.0):
    """(C, gate) of the fixed-shift softmax for n_keys keys and a value bound (host-only)."""
    c, g = ctypes.c_int(), ctypes.c_int()
    st = lib().nbx_decode_fixed_shift_gate(int(n_keys), float(v_max_bound), ctypes.byref(c), ctypes.byref(g))
    _check("nbx_decode_fixed_shift_gate", st)
    return c.value, g.value


# ---------------------------------------------------------------- the block-scaled cache and the pages
# These calls check that every tensor sits on one device, and run there whatever the current device is.
# Their GPU work can be as short as a few microseconds, so the checks keep to a few cheap tensor methods,
# pointers are passed as plain integers and the stream is looked up as a raw handle.
def _one_device(names: str, *tensors) -> int:
    """The index of the CUDA device that all the given tensors (None skipped, the first is one) sit on; contiguous
    all."""
    dev = tensors[0].get_device()
    if dev < 0 or [1 for t in tensors if t is not None and (t.get_device() != dev or not t.is_contiguous())]:
        for name, t in zip(names.split(), tensors):
            if t is None:
                continue
            if t.get_device() < 0:
                raise ValueError(f"{name} must be a CUDA tensor")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.get_device() != dev:
                raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{dev}")
    return dev


def _int32(names: str, *tensors, int32=torch.int32):
    """All int32; the last is the status word, with room for it."""
    if tensors[-1] is not None and not tensors[-1].numel():
        raise ValueError("status has no element")
    if [1 for t in tensors if t is not None and t.dtype is not int32]:
        for name, t in zip(names.split(), tensors):
            if t is not None and t.dtype is not int32:
                raise ValueError(f"{name} must be int32")


def _misfit(names: str, *tensors):
    raise ValueError("shapes do not fit: " + ", ".join(f"{n} {list(t.shape)}" for n, t in zip(names.split(), tensors)
                                                       if t is not None))


def _p(t):
    return 0 if t is None else t.data_ptr()




_calls = {}   # entry point -> its number in nbx_call, and what packs its arguments
_CALLS = ("nbx_paged_kv_append_block_scaled", "nbx_paged_decode_attn_block_scaled", "nbx_paged_decode_attn_modified",
          "nbx_paged_kv_copy_pages", "nbx_paged_kv_fork", "nbx_paged_kv_compact")
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _callable(func: str):
    types = getattr(lib(), func).argtypes
    form = struct.Struct("=" + "".join("d" if t is ctypes.c_float else "q" for t in types))
    _calls[func] = _CALLS.index(func), form.pack
    return _calls[func]


def _run(func: str, dev: int, stream, *args):
    """Calls the entry point on device `dev` and the given (or its current) stream, the last argument."""
    st = _raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)
    call, pack = _calls.get(func) or _callable(func)
    if _current_device() == dev:
        code = _lib.nbx_call(call, pack(*args, st))
    else:
        with torch.cuda.device(dev):
            code = _lib.nbx_call(call, pack(*args, st))
    if code:
        raise NbxError(func, code)


def _pools(k_pool, v_pool, k_scales, v_scales, scaled=False):
    """(num_pages, h_kv, page_tokens, d, positions per scale or 0) of a layer's pools. scaled: the call needs scales."""
    shape = k_pool.shape
    if len(shape) != 4 or shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("k_pool and v_pool [num_pages, h_kv, page_tokens, d] must match")
    num_pages, h_kv, page_tokens, d = shape
    if k_scales is None and v_scales is None and not scaled:
        return num_pages, h_kv, page_tokens, d, 0
    if k_scales is None or v_scales is None:
        raise ValueError("a block-scaled call takes k_scales and v_scales" if scaled else
                         "k_scales and v_scales come together")
    blocks = k_scales.shape
    if k_scales.dtype is not torch.float32 or v_scales.dtype is not torch.float32 or blocks != v_scales.shape or \
            len(blocks) != 3 or blocks[0] != num_pages or blocks[1] != h_kv or blocks[2] < 1 or \
            page_tokens % blocks[2] != 0:
        raise ValueError(f"k_scales {list(blocks)} and v_scales {list(v_scales.shape)} must be fp32 "
                         f"[num_pages, h_kv, page_tokens / scale_tokens] for the pool {list(shape)}")
    if dtype_code(k_pool) != NBX_E4M3:
        raise ValueError("only e4m3 pools have scales")
    return num_pages, h_kv, page_tokens, d, page_tokens // blocks[2]


def nbx_paged_kv_append_block_scaled(new_k: torch.Tensor, new_v: torch.Tensor, k_pool: torch.Tensor,
                                     v_pool: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                                     block_table: torch.Tensor, lens: torch.Tensor, tok_start: torch.Tensor,
                                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """new_k / new_v [n_tok, h_kv, d] (fp32 or bf16): rows tok_start[b] .. tok_start[b + 1] - 1 are sequence
    b's tokens at positions lens[b] and up, quantised into the e4m3 pools and scales [num_pages, h_kv,
    page_tokens / scale_tokens]. lens [batch] and tok_start [batch + 1] int32; lens is not advanced."""
    dev = _one_device("new_k new_v k_pool v_pool k_scales v_scales block_table lens tok_start status", new_k, new_v,
                      k_pool, v_pool, k_scales, v_scales, block_table, lens, tok_start, status)
    _int32("block_table lens tok_start status", block_table, lens, tok_start, status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales, True)
    new, table, batch = new_k.shape, block_table.shape, lens.numel()
    if new != new_v.shape or new_k.dtype != new_v.dtype or len(new) != 3 or new[1] != h_kv or new[2] != d or \
            len(table) != 2 or table[0] != batch or tok_start.numel() != batch + 1:
        _misfit("new_k new_v k_pool block_table lens tok_start", new_k, new_v, k_pool, block_table, lens, tok_start)
    _run("nbx_paged_kv_append_block_scaled", dev, stream, new_k.data_ptr(), new_v.data_ptr(), dtype_code(new_k), new[0],
         h_kv, d, k_pool.data_ptr(), v_pool.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block, num_pages,
         page_tokens, block_table.data_ptr(), table[1], batch, lens.data_ptr(), tok_start.data_ptr(), _p(status))


def nbx_paged_decode_modified_workspace_bytes(batch: int, rows: int, h_q: int, h_kv: int, d: int,
                                              max_seq_len: int) -> int:
    return int(lib().nbx_paged_decode_modified_workspace_bytes(batch, rows, h_q, h_kv, d, max_seq_len))


def nbx_paged_decode_modified_partial_kernel(q_dtype: int, pool_dtype: int, out_dtype: int, rows: int, h_q: int,
                                             h_kv: int, d: int, num_pages: int, page_tokens: int) -> int:
    """The split-partial kernel a modified or block-scaled decode with these sizes runs (PARTIAL_...)."""
    k = lib().nbx_paged_decode_modified_partial_kernel(q_dtype, pool_dtype, out_dtype, rows, h_q, h_kv, d, num_pages,
                                                       page_tokens)
    _check("nbx_paged_decode_modified_partial_kernel", k if k < 0 else 0)
    return k


def _modified_shapes(q, d, block_table, seq_lens, slopes, key_begin, key_end, out, out_dtype, status, stream):
    """The checks the two modified decodes share: (batch, rows, h_q, max_pages, out)."""
    shape, table = q.shape, block_table.shape
    _int32("block_table seq_lens key_begin key_end status", block_table, seq_lens, key_begin, key_end, status)
    if len(shape) != 4 or shape[3] != d or len(table) != 2 or table[0] != shape[0] or seq_lens.numel() != shape[0] or \
            (key_begin is not None and key_begin.shape != shape[:2]) or \
            (key_end is not None and key_end.shape != shape[:2]) or \
            (slopes is not None and slopes.numel() != shape[2]):
        _misfit("q block_table seq_lens slopes key_begin key_end", q, block_table, seq_lens, slopes, key_begin, key_end)
    if slopes is not None and slopes.dtype is not torch.float32:
        raise ValueError("slopes must be fp32")
    if out is None:
        out = _new(shape, out_dtype or torch.float32, q, stream)
    elif out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must be {list(shape)}" + (f" {out_dtype}" if out_dtype else ""))
    return shape[0], shape[1], shape[2], table[1], out


def _workspace(need, like, stream):
    return _new(max(need, 256), torch.uint8, like, stream)


def nbx_paged_decode_attn_block_scaled(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                       k_scales: torch.Tensor, v_scales: torch.Tensor, block_table: torch.Tensor,
                                       seq_lens: torch.Tensor, max_seq_len: int, scale: float, softcap: float = 0.0,
                                       slopes: Optional[torch.Tensor] = None, key_begin: Optional[torch.Tensor] = None,
                                       key_end: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                       out_dtype: Optional[torch.dtype] = None,
                                       workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                       stream=None) -> torch.Tensor:
    """q [batch, rows, h_q, d] (fp32 or bf16) over a block-scaled cache (e4m3 pools, scales [num_pages, h_kv,
    page_tokens / scale_tokens] fp32) -> out [batch, rows, h_q, d], fp32 or bf16 (out's dtype, or out_dtype).
    The score modifications are those of nbx_paged_decode_attn_modified."""
    dev = _one_device("q k_pool v_pool k_scales v_scales block_table seq_lens slopes key_begin key_end out workspace "
                      "status", q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, slopes, key_begin,
                      key_end, out, workspace, status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales, True)
    batch, rows, h_q, max_pages, out = _modified_shapes(q, d, block_table, seq_lens, slopes, key_begin, key_end, out,
                                                        out_dtype, status, stream)
    if workspace is None:
        workspace = _workspace(nbx_paged_decode_modified_workspace_bytes(batch, rows, h_q, h_kv, d, max_seq_len), q,
                               stream)
    _run("nbx_paged_decode_attn_block_scaled", dev, stream, q.data_ptr(), dtype_code(q), batch, rows, h_q, d,
         k_pool.data_ptr(), v_pool.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block, num_pages, h_kv,
         page_tokens, block_table.data_ptr(), max_pages, seq_lens.data_ptr(), int(max_seq_len), float(scale),
         float(softcap), _p(slopes), _p(key_begin), _p(key_end), out.data_ptr(), dtype_code(out),
         workspace.data_ptr(), workspace.nbytes, _p(status))
    return out


def nbx_paged_decode_attn_modified(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                   block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                                   k_scale: float = 1.0, v_scale: float = 1.0, softcap: float = 0.0,
                                   slopes: Optional[torch.Tensor] = None, key_begin: Optional[torch.Tensor] = None,
                                   key_end: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                   out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """nbx_paged_decode_attn with score modifications: a cap (softcap * tanh(z / softcap)), a bias by distance
    (-slopes[h] * |p - j|, slopes [h_q] fp32) and per-row key ranges (key_begin / key_end [batch, rows] int32, by
    default 0 and p + 1: document, prefix and window masks). out [batch, rows, h_q, d] is fp32 or bf16 (out's dtype,
    or out_dtype)."""
    dev = _one_device("q k_pool v_pool block_table seq_lens slopes key_begin key_end out workspace status", q, k_pool,
                      v_pool, block_table, seq_lens, slopes, key_begin, key_end, out, workspace, status)
    num_pages, h_kv, page_tokens, d, _ = _pools(k_pool, v_pool, None, None)
    batch, rows, h_q, max_pages, out = _modified_shapes(q, d, block_table, seq_lens, slopes, key_begin, key_end, out,
                                                        out_dtype, status, stream)
    if workspace is None:
        workspace = _workspace(nbx_paged_decode_modified_workspace_bytes(batch, rows, h_q, h_kv, d, max_seq_len), q,
                               stream)
    _run("nbx_paged_decode_attn_modified", dev, stream, q.data_ptr(), dtype_code(q), batch, rows, h_q, d,
         k_pool.data_ptr(), v_pool.data_ptr(), dtype_code(k_pool), num_pages, h_kv, page_tokens, block_table.data_ptr(),
         max_pages, seq_lens.data_ptr(), int(max_seq_len), float(scale), float(k_scale), float(v_scale), float(softcap),
         _p(slopes), _p(key_begin), _p(key_end), out.data_ptr(), dtype_code(out), workspace.data_ptr(),
         workspace.nbytes, _p(status))
    return out


def nbx_paged_kv_copy_pages(moves: torch.Tensor, n_moves: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                            k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                            status: Optional[torch.Tensor] = None, stream=None) -> None:
    """The first n_moves[0] of moves [max_moves, 3] int32 {source page, destination page, positions}, on one
    layer's pools and, for a block-scaled cache, scales."""
    dev = _one_device("moves n_moves k_pool v_pool k_scales v_scales status", moves, n_moves, k_pool, v_pool, k_scales,
                      v_scales, status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    _int32("moves n_moves status", moves, n_moves, status)
    if moves.dim() != 2 or moves.shape[1] != 3 or n_moves.numel() < 1:
        _misfit("moves n_moves", moves, n_moves)
    _run("nbx_paged_kv_copy_pages", dev, stream, moves.data_ptr(), n_moves.data_ptr(), moves.shape[0],
         k_pool.data_ptr(), v_pool.data_ptr(), dtype_code(k_pool), num_pages, h_kv, page_tokens, d, _p(k_scales),
         _p(v_scales), block, _p(status))


def nbx_paged_kv_fork_workspace_bytes(batch: int, max_pages: int, n_fork: int, num_pages: int) -> int:
    return int(lib().nbx_paged_kv_fork_workspace_bytes(batch, max_pages, n_fork, num_pages))


def nbx_paged_kv_fork(block_table: torch.Tensor, seq_lens: torch.Tensor, fork_src: torch.Tensor,
                      fork_dst: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                      k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                      moves: Optional[torch.Tensor] = None, n_moves: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Rows fork_dst[i] of block_table [batch, max_pages] and seq_lens [batch] become rows fork_src[i] as they
    were (all int32): full pages shared, the last partial page copied to a free one. Returns (moves [n_fork, 3],
    n_moves [1]): the copies made, for nbx_paged_kv_copy_pages on the other layers' pools."""
    dev = _one_device("block_table seq_lens fork_src fork_dst k_pool v_pool k_scales v_scales moves n_moves workspace "
                      "status", block_table, seq_lens, fork_src, fork_dst, k_pool, v_pool, k_scales, v_scales, moves,
                      n_moves, workspace, status)
    _int32("block_table seq_lens fork_src fork_dst moves n_moves status", block_table, seq_lens, fork_src, fork_dst,
           moves, n_moves, status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    n, table = fork_src.numel(), block_table.shape
    # (the call writes all of both; one without a fork or a row writes nothing)
    no_rows = len(table) == 2 and table[0] == 0
    if moves is None:
        moves = _new((n, 3), torch.int32, block_table, stream, -1 if no_rows else None)
    if n_moves is None:
        n_moves = _new(1, torch.int32, block_table, stream, 0 if n == 0 or no_rows else None)
    if len(table) != 2 or seq_lens.numel() != table[0] or fork_dst.numel() != n or moves.shape != (n, 3) or \
            n_moves.numel() < 1:
        _misfit("block_table seq_lens fork_src fork_dst moves n_moves", block_table, seq_lens, fork_src, fork_dst,
                moves, n_moves)
    if workspace is None:
        workspace = _workspace(nbx_paged_kv_fork_workspace_bytes(table[0], table[1], n, num_pages), block_table, stream)
    _run("nbx_paged_kv_fork", dev, stream, block_table.data_ptr(), table[1], seq_lens.data_ptr(), table[0],
         fork_src.data_ptr(), fork_dst.data_ptr(), n, k_pool.data_ptr(), v_pool.data_ptr(), dtype_code(k_pool),
         num_pages, h_kv, page_tokens, d, _p(k_scales), _p(v_scales), block, moves.data_ptr(), n_moves.data_ptr(),
         workspace.data_ptr(), workspace.nbytes, _p(status))
    return moves, n_moves


def nbx_paged_kv_compact_workspace_bytes(num_pages: int) -> int:
    return int(lib().nbx_paged_kv_compact_workspace_bytes(num_pages))


def nbx_paged_kv_compact(block_table: torch.Tensor, seq_lens: torch.Tensor, k_pool: torch.Tensor,
                         v_pool: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                         v_scales: Optional[torch.Tensor] = None, new_block_table: Optional[torch.Tensor] = None,
                         moves: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """The pages in use moved to the lowest ids. Returns (new_block_table, moves [num_pages // 2, 3], counts [2] =
    {moves, pages in use}); new_block_table may be block_table itself. The moves are for
    nbx_paged_kv_copy_pages on the other layers' pools."""
    dev = _one_device("block_table seq_lens k_pool v_pool k_scales v_scales new_block_table moves counts workspace "
                      "status", block_table, seq_lens, k_pool, v_pool, k_scales, v_scales, new_block_table, moves,
                      counts, workspace, status)
    _int32("block_table seq_lens new_block_table moves counts status", block_table, seq_lens, new_block_table, moves,
           counts, status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    table = block_table.shape
    if new_block_table is None:
        new_block_table = _new(table, torch.int32, block_table, stream)
    empty = len(table) == 2 and table[0] == 0   # (such a call writes nothing, any other all of moves and counts)
    if moves is None:
        moves = _new((max(1, num_pages // 2), 3), torch.int32, block_table, stream, -1 if empty else None)
    if counts is None:
        counts = _new(2, torch.int32, block_table, stream, 0 if empty else None)
    if len(table) != 2 or seq_lens.numel() != table[0] or new_block_table.shape != table or moves.dim() != 2 or \
            moves.shape[1] != 3 or counts.numel() < 2:
        _misfit("block_table seq_lens new_block_table moves counts", block_table, seq_lens, new_block_table, moves,
                counts)
    if workspace is None:
        workspace = _workspace(nbx_paged_kv_compact_workspace_bytes(num_pages), block_table, stream)
    _run("nbx_paged_kv_compact", dev, stream, block_table.data_ptr(), new_block_table.data_ptr(), table[1],
         seq_lens.data_ptr(), table[0], k_pool.data_ptr(), v_pool.data_ptr(), dtype_code(k_pool), num_pages, h_kv,
         page_tokens, d, _p(k_scales), _p(v_scales), block, moves.data_ptr(), moves.shape[0], counts.data_ptr(),
         workspace.data_ptr(), workspace.nbytes, _p(status))
    return new_block_table, moves, counts
