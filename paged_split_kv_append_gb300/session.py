"""Device state for one paged decode workload, and its decode step.

A ``PagedDecodeSession`` owns the device buffers a serving loop keeps resident: the K
and V pools, the block table and lengths, the step's queries and new tokens, the
decode workspace, the output and the status word. ``step()`` is one pass of the hot
path through the C ABI: ``nbx_paged_kv_append`` writes the step's new positions into
the pools, then ``nbx_paged_decode_attn`` computes attention for every query row.

With ``scale_tokens`` the pools are a block-scaled cache (E4M3 codes, a scale per block of tokens and
head), appended to by ``nbx_paged_kv_append_block_scaled`` and read by
``nbx_paged_decode_attn_block_scaled``; with score modifications (``set_modifications``) a decode is
``nbx_paged_decode_attn_modified``. ``fork`` and ``compact`` manage the rows and pages of the block table
in place. Nothing here computes: torch provides memory and streams only.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import (NBX_BF16, NBX_E4M3, NBX_F32, _new, nbx_paged_decode_attn, nbx_paged_decode_attn_block_scaled,
               nbx_paged_decode_attn_modified, nbx_paged_decode_modified_workspace_bytes,
               nbx_paged_decode_workspace_bytes_for, nbx_paged_kv_append, nbx_paged_kv_append_block_scaled,
               nbx_paged_kv_compact, nbx_paged_kv_compact_workspace_bytes, nbx_paged_kv_fork,
               nbx_paged_kv_fork_workspace_bytes)

POOL_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


def new_pool(num_pages: int, h_kv: int, page_tokens: int, d: int, dtype: str, device, fill_nan: bool = True):
    """A pool [num_pages, h_kv, page_tokens, d]; e4m3 pools are held as uint8 codes. With
    ``fill_nan`` every position starts as NaN (0x7F for e4m3), so a read of a position the
    pool does not hold shows up in the output."""
    shape = (num_pages, h_kv, page_tokens, d)
    if dtype == "e4m3":
        return torch.full(shape, 0x7F if fill_nan else 0, dtype=torch.uint8, device=device)
    return torch.full(shape, float("nan") if fill_nan else 0.0, dtype=POOL_TORCH[dtype], device=device)


class PagedDecodeSession:
    def __init__(self, *, num_pages: int, h_kv: int, page_tokens: int, d: int, pool_dtype: str, batch: int,
                 rows: int, h_q: int, max_seq_len: int, device, fill_nan: bool = True, q_dtype: str = "bf16",
                 scale_tokens: int = 0, modified: bool = False, out_dtype: torch.dtype = torch.float32):
        """scale_tokens: positions per scale of a block-scaled cache (pool_dtype "e4m3"), 0 for one scale per
        pool. modified: size the workspace for score modifications. out_dtype: fp32, or bf16 for a session that is
        block-scaled or modified."""
        self.device = torch.device(device)
        self.num_pages, self.h_kv, self.page_tokens, self.d = num_pages, h_kv, page_tokens, d
        self.pool_dtype = pool_dtype
        self.batch, self.rows, self.h_q, self.max_seq_len = batch, rows, h_q, max_seq_len
        self.k_pool = new_pool(num_pages, h_kv, page_tokens, d, pool_dtype, self.device, fill_nan)
        self.v_pool = new_pool(num_pages, h_kv, page_tokens, d, pool_dtype, self.device, fill_nan)
        codes = {"f32": NBX_F32, "bf16": NBX_BF16, "e4m3": NBX_E4M3}
        if scale_tokens and (pool_dtype != "e4m3" or page_tokens % scale_tokens):
            raise ValueError("scales belong to e4m3 pools, and a page holds a whole number of their blocks")
        self.k_scales = self.v_scales = None
        if scale_tokens:
            shape = (num_pages, h_kv, page_tokens // scale_tokens)
            self.k_scales = torch.ones(shape, dtype=torch.float32, device=self.device)
            self.v_scales = torch.ones_like(self.k_scales)
        self.modified = modified or scale_tokens > 0
        if out_dtype != torch.float32 and not self.modified:
            raise ValueError("a plain decode's output is fp32")
        ws = nbx_paged_decode_workspace_bytes_for(codes[q_dtype], codes[pool_dtype], batch, rows, h_q, h_kv, d,
                                                  max_seq_len, page_tokens)
        if self.modified:
            ws = nbx_paged_decode_modified_workspace_bytes(batch, rows, h_q, h_kv, d, max_seq_len)
        if ws == 0 and batch > 0:
            raise ValueError("invalid decode sizes")
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=self.device)
        self.out = torch.empty((batch, rows, h_q, d), dtype=out_dtype, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.q = self.block_table = self.seq_lens = None
        self.new_k = self.new_v = self.new_slots = None
        self.held = self.tok_start = None
        self.scale, self.k_scale, self.v_scale = 1.0, 1.0, 1.0
        self.modifications = {}
        self._page_workspaces = []

    # ---------------------------------------------------------------- state
    def _fits(self, call: str, block_scaled: bool) -> None:
        """Refuses a call that does not know of the pools' block scales, or one that needs them."""
        if (self.k_scales is not None) != block_scaled:
            raise ValueError(f"{call} is for a session " + ("with" if block_scaled else "without") + " block scales")

    def append(self, new_k: torch.Tensor, new_v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        self._fits("append", False)
        nbx_paged_kv_append(new_k, new_v, self.k_pool, self.v_pool, slots, self.k_scale, self.v_scale,
                            status=self.status, stream=stream)

    def prefill(self, k_raw: torch.Tensor, v_raw: torch.Tensor, index, slots, chunk_tokens: int = 1 << 18) -> None:
        """Append the tokens k_raw[index] at the given slots, in chunks (index/slots on the host)."""
        self._fits("prefill", False)
        import numpy as np
        index = np.asarray(index)
        slots = np.asarray(slots, dtype=np.int32)
        for lo in range(0, index.size, chunk_tokens):
            hi = min(index.size, lo + chunk_tokens)
            ii = torch.from_numpy(index[lo:hi]).to(k_raw.device)
            kk = k_raw.index_select(0, ii).to(self.device)
            vv = v_raw.index_select(0, ii).to(self.device)
            ss = torch.from_numpy(slots[lo:hi]).to(self.device)
            self.append(kk, vv, ss)

    def set_inputs(self, q: torch.Tensor, block_table, seq_lens, new_k: Optional[torch.Tensor],
                   new_v: Optional[torch.Tensor], new_slots, scale: float, k_scale: float = 1.0,
                   v_scale: float = 1.0) -> None:
        """The step's inputs; host arrays are copied to the device once. (A block-scaled session's scales are its
        blocks', and what its steps append is said by set_new_tokens.)"""
        if self.k_scales is not None and (k_scale != 1.0 or v_scale != 1.0):
            raise ValueError("a session with block scales takes no scale of the pool")
        def dev(x, dtype=None):
            t = x if isinstance(x, torch.Tensor) else torch.as_tensor(x)
            if dtype is not None:
                t = t.to(dtype)
            return t.to(self.device).contiguous()
        self.q = dev(q)
        self.block_table = dev(block_table, torch.int32)
        self.seq_lens = dev(seq_lens, torch.int32)
        self.new_k = None if new_k is None else dev(new_k)
        self.new_v = None if new_v is None else dev(new_v)
        self.new_slots = None if new_slots is None else dev(new_slots, torch.int32)
        self.scale, self.k_scale, self.v_scale = float(scale), float(k_scale), float(v_scale)

    def append_block_scaled(self, new_k: torch.Tensor, new_v: torch.Tensor, held: torch.Tensor,
                            tok_start: torch.Tensor, stream=None) -> None:
        """Rows tok_start[b] .. tok_start[b + 1] - 1 to positions held[b] and up of sequence b (a block-scaled
        cache)."""
        self._fits("append_block_scaled", True)
        nbx_paged_kv_append_block_scaled(new_k, new_v, self.k_pool, self.v_pool, self.k_scales, self.v_scales,
                                         self.block_table, held, tok_start, status=self.status, stream=stream)

    def set_new_tokens(self, new_k: torch.Tensor, new_v: torch.Tensor, held, tok_start) -> None:
        """The tokens a step of a block-scaled session appends; host arrays are copied to the device once."""
        self._fits("set_new_tokens", True)
        def dev(x):
            return torch.as_tensor(x).to(torch.int32).to(self.device).contiguous()
        self.new_k, self.new_v = new_k.to(self.device).contiguous(), new_v.to(self.device).contiguous()
        self.held, self.tok_start = dev(held), dev(tok_start)

    def set_modifications(self, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                          key_begin: Optional[torch.Tensor] = None, key_end: Optional[torch.Tensor] = None) -> None:
        """The score modifications of the decodes from here on (device tensors)."""
        if not self.modified:
            raise ValueError("the session was not made for score modifications")
        self.modifications = dict(softcap=softcap, slopes=slopes, key_begin=key_begin, key_end=key_end)

    # ---------------------------------------------------------------- rows and pages
    def _page_scratch(self, stream) -> torch.Tensor:
        """The workspace of forks (of up to a row each) and compactions. One that a larger table outgrows is kept beside
        its successor: captured graphs, and calls on other streams, may still use it."""
        need = max(nbx_paged_kv_fork_workspace_bytes(*self.block_table.shape, self.batch, self.num_pages),
                   nbx_paged_kv_compact_workspace_bytes(self.num_pages))
        if not self._page_workspaces or self._page_workspaces[-1].numel() < need:
            self._page_workspaces.append(_new(need, torch.uint8, self.block_table, stream))
        return self._page_workspaces[-1]

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        """Rows dst of the block table and the lengths become rows src as they were (int32 device tensors). Returns
        (moves, n_moves)."""
        return nbx_paged_kv_fork(self.block_table, self.seq_lens, src, dst, self.k_pool, self.v_pool, self.k_scales,
                                 self.v_scales, workspace=self._page_scratch(stream), status=self.status, stream=stream)

    def compact(self, stream=None):
        """The pages in use move to the lowest ids, in the block table too. Returns (moves, {moves, pages in use})."""
        return nbx_paged_kv_compact(self.block_table, self.seq_lens, self.k_pool, self.v_pool, self.k_scales,
                                    self.v_scales, new_block_table=self.block_table, workspace=self._page_scratch(stream),
                                    status=self.status, stream=stream)[1:]

    # ---------------------------------------------------------------- the step
    def decode(self, stream=None) -> torch.Tensor:
        if self.k_scales is not None:
            return nbx_paged_decode_attn_block_scaled(self.q, self.k_pool, self.v_pool, self.k_scales, self.v_scales,
                                                      self.block_table, self.seq_lens, self.max_seq_len, self.scale,
                                                      out=self.out, workspace=self.workspace, status=self.status,
                                                      stream=stream, **self.modifications)
        if self.modified:
            return nbx_paged_decode_attn_modified(self.q, self.k_pool, self.v_pool, self.block_table, self.seq_lens,
                                                  self.max_seq_len, self.scale, self.k_scale, self.v_scale,
                                                  out=self.out, workspace=self.workspace, status=self.status,
                                                  stream=stream, **self.modifications)
        return nbx_paged_decode_attn(self.q, self.k_pool, self.v_pool, self.block_table, self.seq_lens,
                                     self.max_seq_len, self.scale, self.k_scale, self.v_scale, out=self.out,
                                     workspace=self.workspace, status=self.status, stream=stream)

    def step(self, stream=None) -> torch.Tensor:
        """Append the step's new positions, then decode: one pass of the hot path."""
        if self.k_scales is not None:
            if self.new_k is not None:
                if self.held is None:
                    raise ValueError("a step of a session with block scales appends what set_new_tokens gives it")
                self.append_block_scaled(self.new_k, self.new_v, self.held, self.tok_start, stream=stream)
        elif self.new_k is not None and self.new_k.shape[0] > 0:
            self.append(self.new_k, self.new_v, self.new_slots, stream=stream)
        return self.decode(stream=stream)

    def status_bits(self) -> int:
        return int(self.status.item())
