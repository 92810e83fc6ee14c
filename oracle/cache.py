"""The block-scaled cache, the score modifications and the page calls, from their definitions
(oracle; test infrastructure only).

Everything is written position by position and page by page in float64 or whole numbers: no tiles, no
bitmaps, no ranks. Notation as in ``oracle.paged``; T = positions per scale of a block-scaled pool.
"""

from __future__ import annotations

import numpy as np

from . import formats, paged

SCALE_LOG2 = 48     # a block's scale is a power of two in [2^-48, 2^48]


def block_scale(amax: float) -> float:
    """The smallest power of two S in [2^-48, 2^48] with amax <= 448 S (at most 2^48)."""
    for e in range(-SCALE_LOG2, SCALE_LOG2 + 1):
        if amax <= formats.E4M3_MAX * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** SCALE_LOG2


def append_block_scaled(codes: np.ndarray, scales: np.ndarray, new: np.ndarray, block_table: np.ndarray,
                        lens, tok_start, T: int) -> None:
    """One pool's append, in place. codes [num_pages, h, P, d] uint8, scales [num_pages, h, P / T] float32,
    new [n_tok, h, d] float32. A block's scale is set by the finite values of its new tokens, and by the scale
    it has when positions of it are held already; held codes follow a scale that grows."""
    P = codes.shape[2]
    for b in range(len(lens)):
        held, n = int(lens[b]), int(tok_start[b + 1]) - int(tok_start[b])
        for first in range(held // T * T, held + n, T):
            if n == 0:
                break
            page = int(block_table[b, first // P])
            in_page = first % P
            lo, hi = max(first, held), min(first + T, held + n)
            x = new[int(tok_start[b]) + lo - held:int(tok_start[b]) + hi - held].astype(np.float64)
            for h in range(codes.shape[1]):
                v = x[:, h]
                a = np.abs(v[np.isfinite(v)])
                need = block_scale(float(a.max()) if a.size else 0.0)
                was = float(scales[page, h, in_page // T])
                s = need if lo == first else max(was, need)
                if lo > first and s > was:
                    old = codes[page, h, in_page:in_page + lo - first]
                    codes[page, h, in_page:in_page + lo - first] = formats.e4m3_encode(
                        (formats.e4m3_decode(old) * (was / s)).astype(np.float32))
                codes[page, h, in_page + lo - first:in_page + hi - first] = formats.e4m3_encode(
                    (v / s).astype(np.float32))
                scales[page, h, in_page // T] = s


def pool_values(pool: np.ndarray, dtype: str, scale: float = 1.0, scales: np.ndarray | None = None) -> np.ndarray:
    """What a pool stands for, float64 [num_pages, h, P, d]."""
    v = formats.decode(pool, dtype) * float(scale)
    if scales is not None:
        v = v * np.repeat(np.asarray(scales, dtype=np.float64), pool.shape[2] // scales.shape[2], axis=2)[..., None]
    return v


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, block_table: np.ndarray, seq_lens, scale: float,
              softcap: float = 0.0, slopes=None, key_begin=None, key_end=None) -> np.ndarray:
    """Attention over pools of values (``pool_values``), float64 [B, R, Hq, D].

    Row r of sequence b sits at p = len - R + r and sees the keys j of [key_begin, key_end) that the sequence
    holds (by default 0 and p + 1): z_j = scale q.k_j; z_j = softcap tanh(z_j / softcap) if softcap > 0;
    z_j -= slopes[h] |p - j|; softmax over the seen keys, times the values. No key seen -> 0."""
    q = np.asarray(q, dtype=np.float64)
    B, R, Hq, D = q.shape
    P, h_kv = k.shape[2], k.shape[1]
    out = np.zeros((B, R, Hq, D))
    for b in range(B):
        n = int(seq_lens[b])
        if n <= 0:
            continue
        pages = np.asarray(block_table[b, : -(-n // P)], dtype=np.int64)
        for h in range(Hq):
            g = paged.kv_head(h, Hq, h_kv)
            K = k[pages, g].reshape(-1, D)[:n]
            V = v[pages, g].reshape(-1, D)[:n]
            for r in range(R):
                p = paged.query_position(n, R, r)
                lo = 0 if key_begin is None else max(0, int(key_begin[b, r]))
                hi = min(n, p + 1 if key_end is None else int(key_end[b, r]))
                if hi <= lo:
                    continue
                z = scale * (K[lo:hi] @ q[b, r, h])
                if softcap > 0:
                    z = softcap * np.tanh(z / softcap)
                if slopes is not None:
                    z = z - float(slopes[h]) * np.abs(p - np.arange(lo, hi))
                w = np.exp(z - z.max())
                out[b, r, h] = (w @ V[lo:hi]) / w.sum()
    return out


def pages_in_use(block_table: np.ndarray, num_pages: int, rows=None) -> set:
    rows = range(block_table.shape[0]) if rows is None else rows
    return {int(p) for b in rows for p in block_table[b] if 0 <= p < num_pages}


def fork(block_table: np.ndarray, seq_lens: np.ndarray, src, dst, P: int, num_pages: int):
    """(table, lens, moves) after the forks; every row is read as it was before them."""
    table, lens = block_table.copy(), np.asarray(seq_lens).copy()
    B, width = block_table.shape
    taken = {}
    for i, (s, d) in enumerate(zip(src, dst)):     # the fork that writes each destination: the first that names it
        if 0 <= s < B and 0 <= d < B and d not in taken:
            taken[d] = i
    read = {s for s, d in zip(src, dst) if 0 <= s < B and 0 <= d < B}
    held = [b for b in range(B) if b not in taken or b in read]
    free = sorted(set(range(num_pages)) - pages_in_use(block_table, num_pages, held))
    moves, seen = [], set()
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (0 <= s < B and 0 <= d < B):
            continue
        first_reader = s not in seen
        seen.add(s)
        if taken.get(d) != i:
            continue
        n = int(seq_lens[s])
        row = np.full(width, -1, dtype=block_table.dtype)
        if not 0 <= n <= width * P:
            table[d], lens[d] = row, 0
            continue
        k = -(-n // P)
        row[:k] = block_table[s, :k]
        if n % P and not (s in taken and first_reader) and 0 <= row[k - 1] < num_pages:
            if not free:
                table[d], lens[d] = -1, 0
                continue
            fresh = free.pop(0)
            moves.append((int(row[k - 1]), fresh, n % P))
            row[k - 1] = fresh
        table[d], lens[d] = row, n
    return table, lens, moves


def compact(block_table: np.ndarray, seq_lens, P: int, num_pages: int):
    """(new table, moves, pages in use)."""
    used = pages_in_use(block_table, num_pages)
    n = len(used)
    src = sorted(p for p in used if p >= n)
    dst = sorted(set(range(n)) - used)
    count = {p: 0 for p in used}
    for b in range(block_table.shape[0]):
        for j, p in enumerate(block_table[b]):
            if 0 <= p < num_pages:
                count[int(p)] = max(count[int(p)], min(P, max(0, int(seq_lens[b]) - j * P)))
    to = dict(zip(src, dst))
    new = np.array([[to.get(int(p), int(p)) for p in row] for row in block_table], dtype=block_table.dtype)
    return new, [(s, d, count[s]) for s, d in zip(src, dst)], n

