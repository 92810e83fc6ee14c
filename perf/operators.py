"""The cache operators of libnbx beyond plain append and decode, as cases to be measured.

Five operators on a paged key/value cache:

- ``append``: new tokens into an 8-bit (E4M3) cache that holds one scale per block of tokens and KV head;
- ``scaled``: split-KV attention over that cache;
- ``modified``: split-KV attention whose scores are capped by a tanh, biased by distance, or masked by
  documents, a prefix or a window;
- ``fork``: rows of the block table that become copies of other rows, sharing their full pages;
- ``compact``: pages in use moved to the lowest ids.

``run`` computes each in elementary torch operations, or, where ``own`` is true, calls the library.
``exact`` computes the first three from their definitions in 64 bits. Lengths, documents and page layouts
follow from the case; values and page ids from the seed.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
ELT = {"f32": 4, "bf16": 2, "e4m3": 1}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------------ cases
def _append(name, batch, lo, hi, new_lo, new_hi, h_kv, d, page, block, new_type, layout):
    return {"name": name, "op": "append", "batch": batch, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi,
            "h_kv": h_kv, "d": d, "page": page, "block": block, "new_type": new_type, "layout": layout}


def _attend(name, op, batch, rows, h_q, h_kv, d, page, lo, hi, pool, q_type, out_type, layout, block=0, cap=0.0,
            slopes=False, mask="causal", span=0):
    return {"name": name, "op": op, "batch": batch, "rows": rows, "h_q": h_q, "h_kv": h_kv, "d": d, "page": page,
            "lo": lo, "hi": hi, "pool": pool, "q_type": q_type, "out_type": out_type, "layout": layout,
            "block": block, "cap": cap, "slopes": slopes, "mask": mask, "span": span}


def _pages(name, op, batch, lo, hi, h_kv, d, page, pool, layout, children=0, spread=2.0):
    return {"name": name, "op": op, "batch": batch, "lo": lo, "hi": hi, "h_kv": h_kv, "d": d, "page": page,
            "pool": pool, "layout": layout, "children": children, "spread": spread}


def listed():
    return [
        # one decode step of 32 sequences: a token each, into blocks that are partly held (latency)
        _append("append step", 32, 512, 8192, 1, 1, 8, 128, 16, 16, "bf16", 1),
        # prompt chunks of 4 sequences, begun inside a block
        _append("append chunks", 4, 1000, 9000, 7001, 8192, 4, 256, 64, 64, "bf16", 2),
        # ordinary single-row decode over the block-scaled cache
        _attend("scaled single row", "scaled", 32, 1, 32, 8, 128, 16, 512, 8192, "e4m3", "bf16", "f32", 3, block=16),
        # a 128-row prompt chunk at the end of a long context: matrix products bound it
        _attend("scaled prompt chunk", "scaled", 1, 128, 24, 4, 256, 64, 32768, 32768, "e4m3", "bf16", "bf16", 5,
                block=64),
        # two short sequences in fp32, capped: the smallest attention call (latency)
        _attend("capped tiny", "modified", 2, 1, 4, 2, 64, 16, 37, 100, "f32", "f32", "f32", 6, cap=30.0),
        # single-row decode of a model whose positions are a bias by distance: 16 sequences from a few
        # positions to very long ones
        _attend("distance ragged", "modified", 16, 1, 32, 8, 128, 16, 1, 131072, "bf16", "bf16", "f32", 24,
                slopes=True),
        # 16-row verify windows at 32768 positions, scores capped
        _attend("capped verify", "modified", 4, 16, 24, 4, 256, 64, 32768, 32768, "bf16", "bf16", "bf16", 8, cap=50.0),
        # a prompt chunk of packed documents: a row sees its own document only
        _attend("documents chunk", "modified", 2, 512, 32, 8, 128, 64, 6000, 16384, "bf16", "bf16", "bf16", 9,
                mask="documents", span=1500),
        # 8 prompts, 8 samples of each
        _pages("fork samples", "fork", 8, 100, 4000, 8, 128, 16, "bf16", 10, children=8),
        # 64 longer prompts on 64-position pages, 16 samples of each
        _pages("fork many", "fork", 64, 1000, 6000, 4, 256, 64, "bf16", 4, children=16),
        # a fragmented small cache
        _pages("compact small", "compact", 12, 20, 900, 8, 128, 16, "bf16", 11),
        # a half-empty cache of a few GB
        _pages("compact large", "compact", 64, 4000, 12000, 4, 256, 64, "bf16", 12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "scaled", "scaled", "modified", "modified", "fork", "compact"])
    layout = rng.randrange(1 << 30)
    if op == "append":
        block = rng.choice([16, 32, 64, 128])
        page = block * rng.choice([1, 2, 4])
        h_kv, d, new_type = rng.randint(1, 8), rng.choice([64, 128, 256]), rng.choice(["bf16", "bf16", "f32"])
        most = 24_000_000 // (h_kv * d * ELT[new_type])
        batch = _log(rng, 1, 64)
        new_hi = _log(rng, 1, max(1, min(8192, most // batch)))
        c = _append("", batch, 0, _log(rng, 16, 8192), rng.choice([0, 1, max(1, new_hi // 2)]) if new_hi > 1 else 1,
                    new_hi, h_kv, d, page, block, new_type, layout)
    elif op in ("scaled", "modified"):
        h_kv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8]), rng.choice([64, 128, 128, 256])
        window = rng.random() < 0.5
        rows = _log(rng, 2, 200) if window else 1
        tensor = rows * group >= 64 and d >= 128
        pool = "e4m3" if op == "scaled" else rng.choice(["bf16", "bf16", "e4m3", "f32"])
        q_type = "bf16" if tensor else rng.choice(["bf16", "f32"])
        out_type = "bf16" if tensor else rng.choice(["f32", "bf16"])
        page = rng.choice([16, 32, 64, 128])
        block = rng.choice([b for b in (16, 32, 64, 128) if page % b == 0]) if op == "scaled" else 0
        batch = _log(rng, 1, 64)
        keys = 400_000_000 // (h_kv * d * ELT[pool] * 2)
        work = 100_000_000_000 // (4 * d * h_kv * group * rows)
        hi = _log(rng, 64, max(64, min(131072, keys // batch, work // batch, 2_000_000_000 // (batch * h_kv * d))))
        mask = rng.choice(["causal", "documents", "prefix", "window"]) if op == "modified" else "causal"
        c = _attend("", op, batch, rows, h_kv * group, h_kv, d, page, 1, hi, pool, q_type, out_type, layout,
                    block=block, cap=rng.choice([0.0, 0.0, 15.0, 50.0]) if op == "modified" else 0.0,
                    slopes=op == "modified" and rng.random() < 0.5, mask=mask,
                    span=0 if mask == "causal" else _log(rng, 1, max(1, hi)))
    else:
        page = rng.choice([16, 32, 64])
        h_kv, d, pool = rng.randint(1, 8), rng.choice([64, 128, 256]), rng.choice(["bf16", "bf16", "f32", "e4m3"])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 16, max(16, min(12000, 500_000_000 // (batch * h_kv * d * ELT[pool]))))
        children = _log(rng, 1, 32) if op == "fork" else 0
        c = _pages("", op, batch, 0, hi, h_kv, d, page, pool, layout, children=children,
                   spread=rng.uniform(1.1, 3.0))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ layouts
def _lens(case):
    """Positions each sequence holds: uniform on [lo, hi], or log-uniform where that spans over 64 times."""
    rng = random.Random(case["layout"])
    lo, hi = case["lo"], case["hi"]
    if hi > 64 * max(lo, 1):
        return [_log(rng, max(lo, 1), hi) for _ in range(case["batch"])]
    return [rng.randint(lo, hi) for _ in range(case["batch"])]


def _new(case):
    rng = random.Random(case["layout"] + 1)
    return [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]


def _ceil(a, b):
    return -(-a // b)


def _intervals(case, lens):
    """Per sequence and row: the first visible key and the one past the last, as lists of tensors' data."""
    R, span, mask = case["rows"], case["span"], case["mask"]
    n = torch.tensor(lens, dtype=torch.int64)[:, None]
    p = n - R + torch.arange(R)[None, :]
    begin, end = torch.zeros_like(p), p + 1
    if mask == "documents":      # documents of `span` positions; a row sees its own up to itself
        begin = (p.clamp(min=0) // span) * span
    elif mask == "prefix":       # the first `span` positions are seen by every row
        end = torch.maximum(p + 1, torch.full_like(p, span))
    elif mask == "window":       # the last `span` positions
        begin = (p + 1 - span).clamp(min=0)
    return begin, end, n, p


def work(case):
    lens = _lens(case)
    op, d, h = case["op"], case["d"], case["h_kv"]
    if op == "append":
        n, T = sum(_new(case)), case["block"]
        blocks = sum(_ceil(a + m, T) - a // T for a, m in zip(lens, _new(case)) if m)
        return {"bytes": 2 * h * (n * d * (ELT[case["new_type"]] + 1) + blocks * 8), "flops": 0}
    if op in ("scaled", "modified"):
        begin, end, n, _ = _intervals(case, lens)
        begin, end = torch.minimum(begin, n), torch.minimum(end.clamp(min=0), n)
        seen = (end - begin).clamp(min=0)
        # keys that some row of the sequence sees: the rows' intervals, united in order of their starts
        order = torch.argsort(begin, dim=1)
        b, e = torch.gather(begin, 1, order), torch.gather(end, 1, order)
        reach = torch.cat([torch.zeros_like(e[:, :1]), torch.cummax(e, 1).values[:, :-1]], 1)
        keys = int((e - torch.maximum(b, reach)).clamp(min=0).sum())
        vectors = case["batch"] * case["rows"] * case["h_q"] * d
        scales = keys / case["block"] * 8 * h if case["block"] else 0
        return {"bytes": keys * h * d * ELT[case["pool"]] * 2 + scales +
                vectors * (ELT[case["q_type"]] + ELT[case["out_type"]]),
                "flops": 4 * d * case["h_q"] * int(seen.sum())}
    P, elt = case["page"], ELT[case["pool"]]
    table = 4 * sum(1 + _ceil(n, P) for n in lens)
    if op == "fork":
        moved = sum(n % P for n in lens) * case["children"]
        return {"bytes": 4 * moved * h * d * elt + table * (1 + case["children"]), "flops": 0}
    live = sum(_ceil(n, P) for n in lens)
    total = int(live * case["spread"]) + 1
    moved = live * (1 - live / total) * (sum(lens) / max(1, live))   # pages are spread evenly over the ids
    return {"bytes": 4 * moved * h * d * elt + 2 * table, "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(lens, rows, page, num_pages, g):
    """A block table of `rows` rows: the first len(lens) hold their pages, ids from one permutation."""
    width = max(1, max(_ceil(n, page) for n in lens))
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    n = torch.tensor([_ceil(n, page) for n in lens], device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < n[:, None]
    table[: len(lens)][held] = ids[: int(n.sum())]
    return table


def _values(shape, g, spread=0.5):
    """Keys or values: normal, with a magnitude of its own for each token."""
    x = torch.randn(shape, generator=g, device=DEV)
    return x.mul_(torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g, device=DEV)))


def _power(amax):
    """The smallest power of two S in [2^-48, 2^48] with amax <= 448 S."""
    f, e = torch.frexp(amax)
    e = torch.where(f > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -48)).clamp(-48, 48)
    return torch.ldexp(torch.ones_like(amax), e)


def _quantise(x, T):
    """Values [num_pages, h, P, d] as E4M3 codes and one power-of-two scale per T positions."""
    n, h, P, d = x.shape
    s = _power(x.view(n, h, P // T, T * d).abs().amax(-1))
    x = x.view(n, h, P // T, T, d) / s[..., None, None]
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(n, h, P, d), s


def prepare(case, seed):
    g = _gen(seed)
    lens = _lens(case)
    op, P, h, d = case["op"], case["page"], case["h_kv"], case["d"]
    s = {"case": case}
    if op == "append":
        new = _new(case)
        total = [a + m for a, m in zip(lens, new)]
        num_pages = max(1, sum(_ceil(n, P) for n in total))
        s["table"] = _table(total, len(lens), P, num_pages, g)
        s["lens"] = _ints(lens)
        s["start"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
        for w in "kv":
            s[w + "_pool"], s[w + "_scales"] = _quantise(_values((num_pages, h, P, d), g), case["block"])
            s["new_" + w] = (2.0 * _values((sum(new), h, d), g)).to(DTYPE[case["new_type"]])
        return s
    if op in ("scaled", "modified"):
        num_pages = max(1, sum(_ceil(n, P) for n in lens))
        s["table"] = _table(lens, len(lens), P, num_pages, g)
        s["lens"] = _ints(lens)
        s["max_len"] = max(lens)
        for w in "kv":
            x = _values((num_pages, h, P, d), g)
            if case["block"]:
                s[w + "_pool"], s[w + "_scales"] = _quantise(x, case["block"])
            elif case["pool"] == "e4m3":
                s[w + "_scale"] = float(x.abs().max()) / 448.0
                s[w + "_pool"] = (x / s[w + "_scale"]).clamp_(-448, 448).to(torch.float8_e4m3fn)
            else:
                s[w + "_pool"] = x.to(DTYPE[case["pool"]])
        shape = (case["batch"], case["rows"], case["h_q"], d)
        s["q"] = torch.randn(shape, generator=g, device=DEV).to(DTYPE[case["q_type"]])
        s["scale"] = 1.0 / math.sqrt(d)
        if case["slopes"]:
            n = case["h_q"]
            s["slopes"] = 2.0 ** (-8.0 * (torch.arange(n, device=DEV, dtype=torch.float32) + 1) / n)
        if case["mask"] != "causal":
            begin, end, _, _ = _intervals(case, lens)
            s["begin"], s["end"] = begin.to(torch.int32).to(DEV), end.to(torch.int32).to(DEV)
        return s
    if op == "fork":
        n = len(lens) * case["children"]
        held = sum(_ceil(x, P) for x in lens)
        num_pages = held + n + 1
        s["table"] = _table(lens, len(lens) + n, P, num_pages, g)
        s["lens"] = _ints(lens + [0] * n)
        s["src"] = _ints([i // case["children"] for i in range(n)])
        s["dst"] = _ints([len(lens) + i for i in range(n)])
        s["moves"] = torch.empty((n, 3), dtype=torch.int32, device=DEV)
        s["counts"] = torch.empty(1, dtype=torch.int32, device=DEV)
    else:
        held = sum(_ceil(x, P) for x in lens)
        num_pages = int(held * case["spread"]) + 1
        s["table"] = _table(lens, len(lens), P, num_pages, g)
        s["new_table"] = torch.empty_like(s["table"])
        s["lens"] = _ints(lens)
        s["moves"] = torch.empty((max(1, num_pages // 2), 3), dtype=torch.int32, device=DEV)
        s["counts"] = torch.empty(2, dtype=torch.int32, device=DEV)
    for w in "kv":
        s[w + "_pool"] = torch.randn((num_pages, h, P, d), generator=g, device=DEV).to(DTYPE[case["pool"]])
    return s


# ------------------------------------------------------------------------------------------------ passes
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _positions(s):
    """Sequence, position and page of every new token."""
    t = torch.arange(s["new_k"].shape[0], device=DEV)
    b = torch.searchsorted(s["start"].long(), t, right=True) - 1
    pos = s["lens"].long()[b] + t - s["start"].long()[b]
    P = s["k_pool"].shape[2]
    return b, pos, s["table"][b, pos // P].long()


def _plain_append(s):
    P, T = s["case"]["page"], s["case"]["block"]
    b, pos, page = _positions(s)
    off, blk = pos % T, (pos % P) // T
    first = torch.maximum(pos - off, s["lens"].long()[b]) - (pos - off)   # the block's first new offset
    leader = off == first
    lp, lb, lf = page[leader], blk[leader], first[leader]
    for w in "kv":
        pool, scales, x = s[w + "_pool"], s[w + "_scales"], s["new_" + w].float()
        n, h, _, d = pool.shape
        amax = x.abs().masked_fill(~torch.isfinite(x), 0.0).amax(-1)                       # [tokens, h]
        most = torch.zeros((n * (P // T), h), device=DEV)
        most.scatter_reduce_(0, (page * (P // T) + blk)[:, None].expand(-1, h), amax, "amax")
        need = _power(most[lp * (P // T) + lb])                                            # [blocks, h]
        old = scales[lp, :, lb]
        grown = torch.where(lf[:, None] > 0, torch.maximum(old, need), need)
        codes = pool.view(torch.uint8).view(n, h, P // T, T, d)
        held = codes[lp, :, lb].view(torch.float8_e4m3fn).float()                          # [blocks, h, T, d]
        again = (held * (old / grown)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        keep = (torch.arange(T, device=DEV)[None, :] < lf[:, None])[:, None, :, None]
        codes[lp, :, lb] = torch.where(keep, again, codes[lp, :, lb])
        scales[lp, :, lb] = grown
        unit = scales[page, :, blk][..., None]
        codes[page, :, blk, off] = (x / unit).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return {k: s[k] for k in ("k_pool", "v_pool", "k_scales", "v_scales")}


def _read(s, w):
    """Keys or values as fp32 [batch, h, positions, d], through the block table."""
    ids = s["table"].clamp(min=0).long()
    pool = s[w + "_pool"]
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    else:
        x = pool[ids].float()
    B, n, h, P, d = x.shape
    if w + "_scales" in s:
        T = s["case"]["block"]
        x.view(B, n, h, P // T, T, d).mul_(s[w + "_scales"][ids][..., None, None])
    elif w + "_scale" in s:
        x.mul_(s[w + "_scale"])
    return x.permute(0, 2, 1, 3, 4).reshape(B, h, n * P, d)


def _plain_attend(s):
    c = s["case"]
    k, v = _read(s, "k"), _read(s, "v")
    B, R, hq, d = s["q"].shape
    h, L = k.shape[1], k.shape[2]
    G = hq // h
    q = s["q"].float().view(B, R, h, G, d).permute(0, 2, 3, 1, 4).reshape(B, h, G * R, d)
    z = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).view(B, h, G, R, L)
    del k
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    n = s["lens"].long()[:, None]
    p = n - R + torch.arange(R, device=DEV)[None, :]
    j = torch.arange(L, device=DEV)
    if c["slopes"]:
        far = (p[:, :, None] - j).abs().float()
        z = z - s["slopes"].view(1, h, G, 1, 1) * far[:, None, None]
    begin, end = (s["begin"].long(), s["end"].long()) if "begin" in s else (torch.zeros_like(p), p + 1)
    sees = (j >= begin[:, :, None]) & (j < torch.minimum(end, n)[:, :, None])
    z = z.masked_fill_(~sees[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m.masked_fill(m == -math.inf, 0.0))
    del z
    out = torch.matmul(e.view(B, h, G * R, L), v.masked_fill_((j >= n)[:, None, :, None], 0.0))
    total = e.sum(-1).view(B, h, G * R, 1)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.view(B, h, G, R, d).permute(0, 3, 1, 2, 4).reshape(B, R, hq, d).to(DTYPE[c["out_type"]])


def _copy(s, src, dst, count):
    """The first `count` positions of pages `src` to pages `dst`."""
    P = s["case"]["page"]
    take = (torch.arange(P, device=DEV)[None, :] < count[:, None])[:, None, :, None]
    for w in "kv":
        pool = s[w + "_pool"]
        x = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        x[dst] = torch.where(take, x[src], x[dst])


def _in_use(table, num_pages):
    use = torch.zeros(num_pages, dtype=torch.bool, device=DEV)
    use[table[table >= 0].long()] = True
    return use


def _plain_fork(s):
    P, table, lens = s["case"]["page"], s["table"], s["lens"]
    src, dst = s["src"].long(), s["dst"].long()
    order = torch.arange(src.numel(), device=DEV)
    over = torch.zeros(table.shape[0], dtype=torch.bool, device=DEV)
    over[dst] = True
    read = torch.zeros_like(over)
    read[src] = True
    free = torch.nonzero(~_in_use(table[~over | read], s["k_pool"].shape[0]))[:, 0]
    n = lens[src].long()
    full, rest = n // P, n % P
    taker = torch.full((table.shape[0],), src.numel(), device=DEV).scatter_reduce(0, src, order, "amin")
    need = (rest > 0) & ~(over[src] & (taker[src] == order))
    rows = table[src]
    rows[torch.arange(table.shape[1], device=DEV)[None, :] >= ((n + P - 1) // P)[:, None]] = -1
    which = torch.nonzero(need)[:, 0]
    at, old = full[which], rows[which, full[which]].long()
    fresh = free[: which.numel()]
    rows[which, at] = fresh.int()
    table[dst] = rows
    lens[dst] = n.int()
    s["moves"].fill_(-1)
    s["moves"][: which.numel()] = torch.stack([old, fresh, rest[which]], 1).int()
    s["counts"].fill_(which.numel())
    _copy(s, old, fresh, rest[which])
    return {k: s[k] for k in ("table", "lens", "moves", "counts", "k_pool", "v_pool")}


def _plain_compact(s):
    P, table, new = s["case"]["page"], s["table"], s["new_table"]
    num_pages = s["k_pool"].shape[0]
    use = _in_use(table, num_pages)
    live = int(use.sum())
    src = torch.nonzero(use[live:])[:, 0] + live
    dst = torch.nonzero(~use[:live])[:, 0]
    here = (table >= 0) & (table < num_pages)
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    fill = (s["lens"].long()[:, None] - col * P).clamp(0, P)
    count = torch.zeros(num_pages, dtype=torch.int64, device=DEV)
    count.scatter_reduce_(0, table[here].long(), fill[here], "amax")
    to = torch.arange(num_pages, device=DEV)
    to[src] = dst
    new.copy_(torch.where(here, to[table.clamp(0, num_pages - 1).long()].int(), table))
    s["moves"].fill_(-1)
    s["moves"][: src.numel()] = torch.stack([src, dst, count[src]], 1).int()
    s["counts"][0], s["counts"][1] = src.numel(), live
    _copy(s, src, dst, count[src])
    return {k: s[k] for k in ("new_table", "moves", "counts", "k_pool", "v_pool")}


def _own_append(s):
    import paged_split_kv_append_gb300 as nbx
    nbx.nbx_paged_kv_append_block_scaled(s["new_k"], s["new_v"], s["k_pool"], s["v_pool"], s["k_scales"],
                                         s["v_scales"], s["table"], s["lens"], s["start"])
    return {k: s[k] for k in ("k_pool", "v_pool", "k_scales", "v_scales")}


def _kept(s):
    """The workspace and output that a serving loop keeps from step to step."""
    import paged_split_kv_append_gb300 as nbx
    if "workspace" not in s:
        c = s["case"]
        size = nbx.nbx_paged_decode_modified_workspace_bytes(c["batch"], c["rows"], c["h_q"], c["h_kv"], c["d"],
                                                             s["max_len"])
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty(s["q"].shape, dtype=DTYPE[c["out_type"]], device=DEV)
    return nbx


def _own_scaled(s):
    nbx = _kept(s)
    return nbx.nbx_paged_decode_attn_block_scaled(s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                                                  s["table"], s["lens"], s["max_len"], s["scale"], out=s["out"],
                                                  workspace=s["workspace"])


def _own_modified(s):
    nbx = _kept(s)
    return nbx.nbx_paged_decode_attn_modified(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["max_len"],
                                              s["scale"], k_scale=s.get("k_scale", 1.0),
                                              v_scale=s.get("v_scale", 1.0), softcap=s["case"]["cap"],
                                              slopes=s.get("slopes"), key_begin=s.get("begin"), key_end=s.get("end"),
                                              out=s["out"], workspace=s["workspace"])


def _own_fork(s):
    import paged_split_kv_append_gb300 as nbx
    if "workspace" not in s:
        size = nbx.nbx_paged_kv_fork_workspace_bytes(*s["table"].shape, s["src"].numel(), s["k_pool"].shape[0])
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    nbx.nbx_paged_kv_fork(s["table"], s["lens"], s["src"], s["dst"], s["k_pool"], s["v_pool"], moves=s["moves"],
                          n_moves=s["counts"], workspace=s["workspace"])
    return {k: s[k] for k in ("table", "lens", "moves", "counts", "k_pool", "v_pool")}


def _own_compact(s):
    import paged_split_kv_append_gb300 as nbx
    if "workspace" not in s:
        size = nbx.nbx_paged_kv_compact_workspace_bytes(s["k_pool"].shape[0])
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    nbx.nbx_paged_kv_compact(s["table"], s["lens"], s["k_pool"], s["v_pool"], new_block_table=s["new_table"],
                             moves=s["moves"], counts=s["counts"], workspace=s["workspace"])
    return {k: s[k] for k in ("new_table", "moves", "counts", "k_pool", "v_pool")}


_run_plain = {"append": _plain_append, "scaled": _plain_attend, "modified": _plain_attend, "fork": _plain_fork,
              "compact": _plain_compact}
_run_own = {"append": _own_append, "scaled": _own_scaled, "modified": _own_modified, "fork": _own_fork,
            "compact": _own_compact}


# ------------------------------------------------------------------------------------------------ 64 bits
def _grid(x):
    """Values rounded to the nearest E4M3 value, ties to the even one, at most 448 in magnitude (float64)."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    step = torch.where(a / step >= 16, step * 2, torch.where(a / step < 8, (step / 2).clamp(min=2.0 ** -9), step))
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    if case["op"] in ("scaled", "modified"):
        return _exact_attend(prepare(case, seed))
    return None


def _exact_append(s):
    P, T = s["case"]["page"], s["case"]["block"]
    table, lens, start = s["table"].tolist(), s["lens"].tolist(), s["start"].tolist()
    got = {}
    for w in "kv":
        codes, scales = s[w + "_pool"].double(), s[w + "_scales"].double()
        h, d = codes.shape[1], codes.shape[3]
        for b, held in enumerate(lens):
            x = s["new_" + w][start[b]:start[b + 1]].double()
            if not x.shape[0]:
                continue
            lo = held // T * T                                   # from the start of the first touched block
            hi = _ceil(held + x.shape[0], T) * T
            at = torch.arange(lo, hi, device=DEV)
            page = torch.tensor(table[b], device=DEV)[at // P]
            was = codes[page, :, at % P]                          # [positions, h, d]
            unit = scales[page[::T], :, (at[::T] % P) // T]       # [blocks, h]
            new = torch.zeros_like(was)
            new[held - lo:held - lo + x.shape[0]] = x
            most = new.view(-1, T, h, d).abs().amax((1, 3))
            need = torch.full_like(most, 2.0 ** -48)
            for e in range(-47, 49):                              # the smallest power of two that holds it
                need = torch.where(most > 448.0 * 2.0 ** (e - 1), torch.full_like(need, 2.0 ** e), need)
            first = torch.arange(0, hi - lo, T, device=DEV) >= held - lo
            to = torch.where(first[:, None], need, torch.maximum(need, unit))
            by = to.repeat_interleave(T, 0)[..., None]
            old = _grid(was * (unit.repeat_interleave(T, 0)[..., None] / by))
            fresh = _grid(new / by)
            where = (at - lo)[:, None, None]
            val = torch.where(where < held - lo, old, torch.where(where < held - lo + x.shape[0], fresh, was))
            codes[page, :, at % P] = val
            scales[page[::T], :, (at[::T] % P) // T] = to
        got[w + "_pool"], got[w + "_scales"] = codes, scales
    return got


def _exact_attend(s):
    c = s["case"]
    B, R, hq, d = s["q"].shape
    h, P = c["h_kv"], c["page"]
    out = torch.zeros((B, R, hq, d), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, : _ceil(n, P)].long()
        at = torch.arange(n, device=DEV)
        p = n - R + torch.arange(R, device=DEV)
        lo = s["begin"][b].long() if "begin" in s else torch.zeros_like(p)
        hi = (s["end"][b].long() if "end" in s else p + 1).clamp(max=n)
        dark = (at < lo[:, None]) | (at >= hi[:, None])
        for i in range(h):
            kv = []
            for w in "kv":
                pool = s[w + "_pool"]
                x = pool.view(torch.uint8)[ids, i].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[ids, i]
                x = x.double()
                if c["block"]:
                    x = x * s[w + "_scales"][ids, i].double().repeat_interleave(c["block"], 1)[..., None]
                kv.append(x.reshape(-1, d)[:n] * s.get(w + "_scale", 1.0))
            heads = slice(i * (hq // h), (i + 1) * (hq // h))
            z = torch.einsum("rgd,jd->rgj", s["q"][b, :, heads].double(), kv[0]) * s["scale"]
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["slopes"]:
                z = z - s["slopes"][heads].double()[None, :, None] * (p[:, None] - at).abs()[:, None].double()
            a = torch.softmax(z.masked_fill(dark[:, None], -math.inf), -1).nan_to_num(0.0)
            out[b, :, heads] = torch.einsum("rgj,jd->rgd", a, kv[1])
    return out
