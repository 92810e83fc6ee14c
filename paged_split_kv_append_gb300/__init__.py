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
    "nbx_paged_decode_modified_workspace_bytes", "nbx_paged_decode_modified_partial_kernel", "nbx_paged_kv_copy_pages", "nbx_paged_kv_fork",
    "nbx_paged_kv_fork_workspace_bytes", "nbx_paged_kv_compact", "nbx_paged_kv_compact_workspace_bytes",
    "dtype_code",
    "DEV_BAD_SLOT", "DEV_BAD_PAGE", "DEV_BAD_LEN", "DEV_TIMEOUT", "DEV_BAD_SCALE", "DEV_BAD_ROW", "DEV_NO_PAGE",
]

NBX_F32, NBX_BF16, NBX_E4M3 = 0, 1, 2
DEV_BAD_SLOT, DEV_BAD_PAGE, DEV_BAD_LEN, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEV_BAD_SCALE, DEV_BAD_ROW, DEV_NO_PAGE = 0x10, 0x20, 0x40
PARTIAL_SIMT, PARTIAL_TCGEN05, PARTIAL_TCGEN05_FP8 = 0, 1, 2

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
    l.nbx_paged_decode_attn_block_scaled.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, i32, i32, i32, i32, vp,
                                                     i32, vp, i32, f32, f32, vp, vp, vp, vp, i32, vp, sz, vp, vp]
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
        out = torch.empty((batch, rows, h_q, d), dtype=torch.float32, device=q.device)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_pool), batch, rows, h_q, h_kv, d,
                                                max_seq_len, page_tokens)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
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
        out = torch.empty((batch, rows, h_q, d), dtype=torch.float32, device=q.device)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_pool), batch, rows, h_q, h_kv, d,
                                                max_seq_len, page_tokens)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
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
        out = torch.empty((batch, rows, h_q, d), dtype=torch.float32, device=q.device)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_cache), batch, rows, h_q, h_kv, d,
                                                max_seq_len, capacity)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
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
        out = torch.empty((n_rows, d), dtype=torch.float32, device=acc_part.device)
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
    q_norm = torch.empty((batch, rows, h_q), dtype=torch.float32, device=q.device)
    kv_max = torch.empty((batch, h_kv, 2), dtype=torch.float32, device=q.device)
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
        out = torch.empty((batch, rows, h_q, d), dtype=torch.float32, device=q.device)
    _cuda_contig("out", out)
    need = nbx_paged_decode_workspace_bytes_for(dtype_code(q), dtype_code(k_pool), batch, rows, h_q, h_kv, d,
                                                max_seq_len, page_tokens)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
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
class _Device:
    """The device of a call's tensors, made current for the call; the stream defaults to its current one."""

    def __init__(self, **tensors):
        self.dev = None
        for n, t in tensors.items():
            if t is None:
                continue
            _cuda_contig(n, t)
            if self.dev is None:
                self.dev = t.device
            elif t.device != self.dev:
                raise ValueError(f"{n} is on {t.device}, not on {self.dev}")
        self.back = None

    def stream(self, stream) -> ctypes.c_void_p:
        return _stream(torch.cuda.current_stream(self.dev) if stream is None else stream)

    def __enter__(self):
        if torch.cuda.current_device() != self.dev.index:
            self.back = torch.cuda.current_device()
            torch.cuda.set_device(self.dev)
        return self

    def __exit__(self, *exc):
        if self.back is not None:
            torch.cuda.set_device(self.back)


def _int32(shape_ok: bool = True, **tensors):
    for n, t in tensors.items():
        if t is not None and t.dtype != torch.int32:
            raise ValueError(f"{n} must be int32")
    if not shape_ok:
        raise ValueError("shapes do not fit: " + ", ".join(f"{n} {list(t.shape)}" for n, t in tensors.items()
                                                           if t is not None))


def _pools(k_pool, v_pool, k_scales, v_scales):
    """(num_pages, h_kv, page_tokens, d, positions per scale or 0) of a layer's pools."""
    if k_pool.dim() != 4 or k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("k_pool and v_pool [num_pages, h_kv, page_tokens, d] must match")
    num_pages, h_kv, page_tokens, d = k_pool.shape
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales and v_scales come together")
    if k_scales is None:
        return num_pages, h_kv, page_tokens, d, 0
    if k_scales.dtype != torch.float32 or v_scales.dtype != torch.float32 or k_scales.shape != v_scales.shape or \
            k_scales.dim() != 3 or tuple(k_scales.shape[:2]) != (num_pages, h_kv) or k_scales.shape[2] < 1 or \
            page_tokens % k_scales.shape[2] != 0:
        raise ValueError(f"k_scales {list(k_scales.shape)} and v_scales {list(v_scales.shape)} must be fp32 "
                         f"[num_pages, h_kv, page_tokens / scale_tokens] for the pool {list(k_pool.shape)}")
    if dtype_code(k_pool) != NBX_E4M3:
        raise ValueError("only e4m3 pools have scales")
    return num_pages, h_kv, page_tokens, d, page_tokens // k_scales.shape[2]


def nbx_paged_kv_append_block_scaled(new_k: torch.Tensor, new_v: torch.Tensor, k_pool: torch.Tensor,
                                     v_pool: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                                     block_table: torch.Tensor, lens: torch.Tensor, tok_start: torch.Tensor,
                                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """new_k / new_v [n_tok, h_kv, d] (fp32 or bf16): rows tok_start[b] .. tok_start[b + 1] - 1 are sequence
    b's tokens at positions lens[b] and up, quantised into the e4m3 pools and scales [num_pages, h_kv,
    page_tokens / scale_tokens]. lens [batch] and tok_start [batch + 1] int32; lens is not advanced."""
    dv = _Device(new_k=new_k, new_v=new_v, k_pool=k_pool, v_pool=v_pool, k_scales=k_scales, v_scales=v_scales,
                 block_table=block_table, lens=lens, tok_start=tok_start, status=status)
    if new_k.dim() != 3 or new_k.shape != new_v.shape or new_k.dtype != new_v.dtype:
        raise ValueError("new_k and new_v [n_tok, h_kv, d] must match")
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    n_tok = new_k.shape[0]
    if tuple(new_k.shape[1:]) != (h_kv, d):
        raise ValueError(f"new {list(new_k.shape)} does not fit the pool {list(k_pool.shape)}")
    batch = lens.numel()
    _int32(block_table.dim() == 2 and block_table.shape[0] == batch and tok_start.numel() == batch + 1,
           block_table=block_table, lens=lens, tok_start=tok_start, status=status)
    with dv:
        st = lib().nbx_paged_kv_append_block_scaled(
            _ptr(new_k), _ptr(new_v), dtype_code(new_k), n_tok, h_kv, d, _ptr(k_pool), _ptr(v_pool), _ptr(k_scales),
            _ptr(v_scales), block, num_pages, page_tokens, _ptr(block_table), block_table.shape[1], batch, _ptr(lens),
            _ptr(tok_start), _ptr(status), dv.stream(stream))
    _check("nbx_paged_kv_append_block_scaled", st)


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


def _modified_call(dv, q, k_pool, block_table, seq_lens, max_seq_len, slopes, key_begin, key_end, out, out_dtype,
                   workspace, status):
    """The shapes and types the two modified decodes share: (out, workspace, workspace bytes)."""
    if q.dim() != 4:
        raise ValueError("q must be [batch, rows, h_q, d]")
    batch, rows, h_q, d = q.shape
    _int32(block_table.dim() == 2 and block_table.shape[0] == batch and seq_lens.numel() == batch and
           all(k is None or tuple(k.shape) == (batch, rows) for k in (key_begin, key_end)), block_table=block_table,
           seq_lens=seq_lens, key_begin=key_begin, key_end=key_end, status=status)
    if k_pool.shape[3] != d:
        raise ValueError(f"q {list(q.shape)} does not fit the pool {list(k_pool.shape)}")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.numel() != h_q):
        raise ValueError("slopes must be fp32 [h_q]")
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=dv.dev)
    elif out.shape != q.shape or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must be {list(q.shape)}" + (f" {out_dtype}" if out_dtype else ""))
    if workspace is None:
        need = nbx_paged_decode_modified_workspace_bytes(batch, rows, h_q, k_pool.shape[1], d, max_seq_len)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dv.dev)
    return out, workspace, workspace.numel() * workspace.element_size()


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
    dv = _Device(q=q, k_pool=k_pool, v_pool=v_pool, k_scales=k_scales, v_scales=v_scales, block_table=block_table,
                 seq_lens=seq_lens, slopes=slopes, key_begin=key_begin, key_end=key_end, out=out, workspace=workspace,
                 status=status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    out, workspace, ws_bytes = _modified_call(dv, q, k_pool, block_table, seq_lens, max_seq_len, slopes, key_begin,
                                              key_end, out, out_dtype, workspace, status)
    batch, rows, h_q, _ = q.shape
    with dv:
        st = lib().nbx_paged_decode_attn_block_scaled(
            _ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(v_scales), block,
            num_pages, h_kv, page_tokens, _ptr(block_table), block_table.shape[1], _ptr(seq_lens), int(max_seq_len),
            float(scale), float(softcap), _ptr(slopes), _ptr(key_begin), _ptr(key_end), _ptr(out), dtype_code(out),
            _ptr(workspace), ws_bytes, _ptr(status), dv.stream(stream))
    _check("nbx_paged_decode_attn_block_scaled", st)
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
    dv = _Device(q=q, k_pool=k_pool, v_pool=v_pool, block_table=block_table, seq_lens=seq_lens, slopes=slopes,
                 key_begin=key_begin, key_end=key_end, out=out, workspace=workspace, status=status)
    num_pages, h_kv, page_tokens, d, _ = _pools(k_pool, v_pool, None, None)
    out, workspace, ws_bytes = _modified_call(dv, q, k_pool, block_table, seq_lens, max_seq_len, slopes, key_begin,
                                              key_end, out, out_dtype, workspace, status)
    batch, rows, h_q, _ = q.shape
    with dv:
        st = lib().nbx_paged_decode_attn_modified(
            _ptr(q), dtype_code(q), batch, rows, h_q, d, _ptr(k_pool), _ptr(v_pool), dtype_code(k_pool), num_pages, h_kv,
            page_tokens, _ptr(block_table), block_table.shape[1], _ptr(seq_lens), int(max_seq_len), float(scale),
            float(k_scale), float(v_scale), float(softcap), _ptr(slopes), _ptr(key_begin), _ptr(key_end), _ptr(out),
            dtype_code(out), _ptr(workspace), ws_bytes, _ptr(status), dv.stream(stream))
    _check("nbx_paged_decode_attn_modified", st)
    return out


def nbx_paged_kv_copy_pages(moves: torch.Tensor, n_moves: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                            k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                            status: Optional[torch.Tensor] = None, stream=None) -> None:
    """The first n_moves[0] of moves [max_moves, 3] int32 {source page, destination page, positions}, on one
    layer's pools and, for a block-scaled cache, scales."""
    dv = _Device(moves=moves, n_moves=n_moves, k_pool=k_pool, v_pool=v_pool, k_scales=k_scales, v_scales=v_scales,
                 status=status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    _int32(moves.dim() == 2 and moves.shape[1] == 3 and n_moves.numel() >= 1, moves=moves, n_moves=n_moves,
           status=status)
    with dv:
        st = lib().nbx_paged_kv_copy_pages(_ptr(moves), _ptr(n_moves), moves.shape[0], _ptr(k_pool), _ptr(v_pool),
                                           dtype_code(k_pool), num_pages, h_kv, page_tokens, d, _ptr(k_scales),
                                           _ptr(v_scales), block, _ptr(status), dv.stream(stream))
    _check("nbx_paged_kv_copy_pages", st)


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
    dv = _Device(block_table=block_table, seq_lens=seq_lens, fork_src=fork_src, fork_dst=fork_dst, k_pool=k_pool,
                 v_pool=v_pool, k_scales=k_scales, v_scales=v_scales, moves=moves, n_moves=n_moves,
                 workspace=workspace, status=status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    n = fork_src.numel()
    if moves is None:
        moves = torch.full((n, 3), -1, dtype=torch.int32, device=dv.dev)
    if n_moves is None:
        n_moves = torch.zeros(1, dtype=torch.int32, device=dv.dev)
    _int32(block_table.dim() == 2 and block_table.shape[0] == seq_lens.numel() and fork_dst.numel() == n and
           tuple(moves.shape) == (n, 3) and n_moves.numel() >= 1, block_table=block_table, seq_lens=seq_lens,
           fork_src=fork_src, fork_dst=fork_dst, moves=moves, n_moves=n_moves, status=status)
    batch, max_pages = block_table.shape
    if workspace is None:
        workspace = torch.empty(max(nbx_paged_kv_fork_workspace_bytes(batch, max_pages, n, num_pages), 256),
                                dtype=torch.uint8, device=dv.dev)
    with dv:
        st = lib().nbx_paged_kv_fork(_ptr(block_table), max_pages, _ptr(seq_lens), batch, _ptr(fork_src),
                                     _ptr(fork_dst), n, _ptr(k_pool), _ptr(v_pool), dtype_code(k_pool), num_pages,
                                     h_kv, page_tokens, d, _ptr(k_scales), _ptr(v_scales), block, _ptr(moves),
                                     _ptr(n_moves), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _ptr(status), dv.stream(stream))
    _check("nbx_paged_kv_fork", st)
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
    dv = _Device(block_table=block_table, seq_lens=seq_lens, k_pool=k_pool, v_pool=v_pool, k_scales=k_scales,
                 v_scales=v_scales, new_block_table=new_block_table, moves=moves, counts=counts, workspace=workspace,
                 status=status)
    num_pages, h_kv, page_tokens, d, block = _pools(k_pool, v_pool, k_scales, v_scales)
    if new_block_table is None:
        new_block_table = torch.empty_like(block_table)
    if moves is None:
        moves = torch.full((max(1, num_pages // 2), 3), -1, dtype=torch.int32, device=dv.dev)
    if counts is None:
        counts = torch.zeros(2, dtype=torch.int32, device=dv.dev)
    _int32(block_table.dim() == 2 and block_table.shape[0] == seq_lens.numel() and
           new_block_table.shape == block_table.shape and moves.dim() == 2 and moves.shape[1] == 3 and
           counts.numel() >= 2, block_table=block_table, seq_lens=seq_lens, new_block_table=new_block_table,
           moves=moves, counts=counts, status=status)
    if workspace is None:
        workspace = torch.empty(max(nbx_paged_kv_compact_workspace_bytes(num_pages), 256), dtype=torch.uint8,
                                device=dv.dev)
    with dv:
        st = lib().nbx_paged_kv_compact(_ptr(block_table), _ptr(new_block_table), block_table.shape[1],
                                        _ptr(seq_lens), block_table.shape[0], _ptr(k_pool), _ptr(v_pool),
                                        dtype_code(k_pool), num_pages, h_kv, page_tokens, d, _ptr(k_scales),
                                        _ptr(v_scales), block, _ptr(moves), moves.shape[0], _ptr(counts),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                                        dv.stream(stream))
    _check("nbx_paged_kv_compact", st)
    return new_block_table, moves, counts
