"""Operators of a serving loop around the paged cache, as cases to be measured.

- ``rotate``: new tokens' queries and keys turned by their positions, keys and values appended to the paged
  cache on the way;
- ``prompt``: causal attention over whole prompts, packed one behind the other, with grouped heads;
- ``shared``: decode attention for sequences that share a long prefix of the cache, computed once for each
  group of them.

``run`` computes each in elementary torch operations, or, where ``own`` is true, calls the library. ``exact``
computes them from their definitions in 64 bits. Lengths and groups follow from the case; values, positions'
pages and page ids from the seed.
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
def _rotate(name, tokens, runs, far, h_q, h_kv, d, turned, paired, page, new_type, pool, layout):
    """`tokens` new tokens in `runs` runs of consecutive positions below `far`; the first `turned` of d elements are
    turned, halves against each other or (paired) neighbours."""
    return {"name": name, "op": "rotate", "tokens": tokens, "runs": runs, "far": far, "h_q": h_q, "h_kv": h_kv, "d": d,
            "turned": turned, "paired": paired, "page": page, "new_type": new_type, "pool": pool, "layout": layout}


def _prompt(name, batch, lo, hi, h_q, h_kv, d, layout):
    return {"name": name, "op": "prompt", "batch": batch, "lo": lo, "hi": hi, "h_q": h_q, "h_kv": h_kv, "d": d,
            "layout": layout}


def _shared(name, groups, members_lo, members_hi, shared_lo, shared_hi, own_lo, own_hi, rows, h_q, h_kv, d, page, pool,
            out_type, layout):
    """Groups of sequences: a prefix that all of a group share, then positions of each one's own."""
    return {"name": name, "op": "shared", "groups": groups, "members_lo": members_lo, "members_hi": members_hi,
            "shared_lo": shared_lo, "shared_hi": shared_hi, "own_lo": own_lo, "own_hi": own_hi, "rows": rows,
            "h_q": h_q, "h_kv": h_kv, "d": d, "page": page, "pool": pool, "out_type": out_type, "layout": layout}


def listed():
    return [
        # one decode step of 32 sequences: a token each (latency)
        _rotate("rotate step", 32, 32, 8192, 32, 8, 128, 128, False, 16, "bf16", "bf16", 1),
        # the packed prompts of a batch, before their attention
        _rotate("rotate prompts", 16384, 9, 8192, 32, 8, 128, 128, False, 64, "bf16", "bf16", 2),
        # chunks of long documents into an 8-bit cache; a quarter of each head is turned, neighbours in pairs
        _rotate("rotate partly e4m3", 8001, 4, 131072, 24, 4, 256, 64, True, 64, "bf16", "e4m3", 3),
        # a single short question (latency)
        _prompt("prompt question", 1, 17, 17, 32, 8, 128, 4),
        # a batch of questions of a few tokens up to a few thousand
        _prompt("prompt packed", 16, 1, 4096, 32, 8, 128, 5),
        # a few documents, wide heads in groups of six
        _prompt("prompt wide heads", 3, 2000, 4500, 24, 4, 256, 6),
        # narrow heads, each with keys of its own
        _prompt("prompt narrow heads", 8, 700, 1700, 16, 16, 64, 7),
        # one long document
        _prompt("prompt long", 1, 16384, 16384, 32, 8, 128, 8),
        # four answers to a question begun (latency)
        _shared("shared few", 1, 4, 4, 500, 520, 1, 40, 1, 32, 8, 128, 16, "bf16", "f32", 9),
        # 64 users behind one system prompt
        _shared("shared system prompt", 1, 64, 64, 8192, 8192, 10, 600, 1, 32, 8, 128, 16, "bf16", "bf16", 10),
        # samples of several documents, verified four tokens at a time
        _shared("shared verify", 5, 5, 12, 6000, 20000, 4, 700, 4, 24, 4, 256, 64, "bf16", "bf16", 11),
        # 32 readers of one long document in an 8-bit cache
        _shared("shared long e4m3", 1, 32, 32, 65536, 65536, 30, 2000, 1, 32, 8, 128, 64, "e4m3", "bf16", 12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "prompt", "shared", "shared"])
    layout = rng.randrange(1 << 30)
    h_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8])
    d = rng.choice([64, 128, 128, 256])
    if op == "rotate":
        new_type = rng.choice(["bf16", "bf16", "f32"])
        most = 200_000_000 // (h_kv * (2 * group + 4) * d * ELT[new_type])
        tokens = _log(rng, 1, min(20000, most))
        runs = min(tokens, _log(rng, 1, 64))
        c = _rotate("", tokens, runs, _log(rng, max(64, tokens), 131072), h_kv * group, h_kv, d,
                    rng.choice([d, d, d // 2, d // 4]), rng.random() < 0.4, rng.choice([16, 32, 64, 128]), new_type,
                    rng.choice(["bf16", "bf16", "e4m3", "f32"]), layout)
    elif op == "prompt":
        batch = _log(rng, 1, 64)
        # the plain form holds every pair of a padded batch
        most = math.isqrt(min(8_000_000_000, 1_000_000_000_000 // d) // (batch * h_kv * group))
        hi = _log(rng, 1, max(1, min(16384, most)))
        c = _prompt("", batch, rng.choice([1, max(1, hi // 2)]), hi, h_kv * group, h_kv, d, layout)
    else:
        pool = rng.choice(["bf16", "bf16", "e4m3"])
        rows = rng.choice([1, 1, 1, 2, 4, 8])
        groups = _log(rng, 1, 8)
        members = _log(rng, 2, max(2, 64 // groups))
        # the plain form holds every sequence's keys of its own, in 32 bits
        most = 1_500_000_000 // (groups * members * h_kv * d)
        pairs = 2_000_000_000 // (groups * members * rows * h_kv * group)
        hi = _log(rng, 64, max(64, min(65536, most, pairs)))
        own_hi = _log(rng, rows, max(rows, min(2048, hi)))
        c = _shared("", groups, max(1, members // 2), members, max(1, hi // 3), hi, rows, own_hi, rows, h_kv * group,
                    h_kv, d, rng.choice([16, 32, 64, 128]), pool, rng.choice(["bf16", "bf16", "f32"]), layout)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ layouts
def _ceil(a, b):
    return -(-a // b)


def _runs(case):
    """(first position, tokens) of each run of consecutive positions."""
    rng = random.Random(case["layout"])
    n, r = case["tokens"], case["runs"]
    cuts = sorted(rng.sample(range(1, n), r - 1)) if r > 1 else []
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    return [(rng.randint(0, max(0, case["far"] - m)), m) for m in sizes]


def _lens(case):
    """Tokens of each prompt: uniform on [lo, hi], or log-uniform where that spans over 64 times."""
    rng = random.Random(case["layout"])
    lo, hi = case["lo"], case["hi"]
    if hi > 64 * lo:
        return [_log(rng, lo, hi) for _ in range(case["batch"])]
    return [rng.randint(lo, hi) for _ in range(case["batch"])]


def _groups(case):
    """Per group: the positions shared (whole pages) and each member's length."""
    rng = random.Random(case["layout"])
    P, got = case["page"], []
    for _ in range(case["groups"]):
        n = rng.randint(case["shared_lo"], case["shared_hi"])
        members = rng.randint(case["members_lo"], case["members_hi"])
        # what a fork shares: the full pages; the rest of the prefix is each one's own copy
        got.append((n // P * P, [n + rng.randint(case["own_lo"], case["own_hi"]) for _ in range(members)]))
    return got


def work(case):
    d, h, hq = case["d"], case["h_kv"], case["h_q"]
    if case["op"] == "rotate":
        n, runs = case["tokens"], _runs(case)
        rows = len(set().union(*(range(a, a + m) for a, m in runs)))   # rows of the tables that are read
        e, p = ELT[case["new_type"]], ELT[case["pool"]]
        return {"bytes": n * d * (2 * hq * e + 2 * h * (e + p)) + rows * case["turned"] * 4 + 8 * n,
                "flops": 3 * n * case["turned"] * (hq + h)}
    if case["op"] == "prompt":
        lens = _lens(case)
        return {"bytes": sum(lens) * d * 2 * (2 * hq + 2 * h), "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    R = case["rows"]
    keys = pairs = count = 0
    for shared, lens in _groups(case):
        keys += shared + sum(n - shared for n in lens)
        pairs += sum(n * R - R * (R - 1) // 2 for n in lens)
        count += len(lens)
    return {"bytes": keys * h * d * ELT[case["pool"]] * 2 + count * R * hq * d * (2 + ELT[case["out_type"]]),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _values(shape, g, spread=0.5):
    """Keys or values: normal, with a magnitude of its own for each token."""
    x = torch.randn(shape, generator=g, device=DEV)
    return x.mul_(torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g, device=DEV)))


def _pool(shape, pool, g):
    """A pool of the given type and its scale."""
    x = _values(shape, g)
    if pool != "e4m3":
        return x.to(DTYPE[pool]), 1.0
    scale = float(x.abs().max()) / 448.0
    return x.div_(scale).clamp_(-448, 448).to(DTYPE[pool]), scale


def prepare(case, seed):
    g = _gen(seed)
    h, hq, d = case["h_kv"], case["h_q"], case["d"]
    s = {"case": case}
    if case["op"] == "rotate":
        n, P = case["tokens"], case["page"]
        runs = _runs(case)
        s["positions"] = torch.cat([torch.arange(a, a + m, dtype=torch.int32) for a, m in runs]).to(DEV)
        # each run goes to pages of its own
        pages = [a // P for a, _ in runs]
        held = [_ceil(a + m, P) - a // P for a, m in runs]
        num_pages = sum(held) + 3
        ids = torch.randperm(num_pages, generator=g, device=DEV)
        base = torch.tensor([sum(held[:i]) - pages[i] for i in range(len(runs))], device=DEV)
        base = base.repeat_interleave(torch.tensor([m for _, m in runs], device=DEV))
        at = s["positions"].long()
        s["slots"] = (ids[base + at // P] * P + at % P).to(torch.int32)
        half = case["turned"] // 2
        angle = torch.arange(case["far"], dtype=torch.float64, device=DEV)[:, None] * \
            10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # queries, keys and values as one projection leaves them
        x = torch.randn((n, hq + 2 * h, d), generator=g, device=DEV).to(DTYPE[case["new_type"]])
        s["q"], s["new_k"], s["new_v"] = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
        for w in "kv":
            s[w + "_pool"] = torch.zeros((num_pages, h, P, d), device=DEV).to(DTYPE[case["pool"]])
            s[w + "_scale"] = 0.015 if case["pool"] == "e4m3" else 1.0
        s["q_out"] = torch.empty((n, hq, d), dtype=s["q"].dtype, device=DEV)
        return s
    if case["op"] == "prompt":
        lens = _lens(case)
        n = sum(lens)
        s["start"] = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["longest"] = max(lens)
        s["q"] = torch.randn((n, hq, d), generator=g, device=DEV).to(torch.bfloat16)
        s["k"] = _values((n, h, d), g).to(torch.bfloat16)
        s["v"] = _values((n, h, d), g).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty_like(s["q"])
        return s
    P, R = case["page"], case["rows"]
    groups = _groups(case)
    lens = [n for _, members in groups for n in members]
    num_pages = sum(a // P + sum(_ceil(n, P) - a // P for n in members) for a, members in groups)
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), _ceil(max(lens), P)), -1, dtype=torch.int32, device=DEV)
    b = at = 0
    for a, members in groups:
        common = ids[at:at + a // P]
        at += a // P
        for n in members:
            more = _ceil(n, P) - a // P
            table[b, :a // P] = common
            table[b, a // P:a // P + more] = ids[at:at + more]
            at += more
            b += 1
    s["table"], s["lens"], s["max_len"] = table, _ints(lens), max(lens)
    s["start"] = _ints([sum(len(m) for _, m in groups[:i]) for i in range(len(groups) + 1)])
    s["shared"] = _ints([a for a, _ in groups])
    for w in "kv":
        s[w + "_pool"], s[w + "_scale"] = _pool((num_pages, h, P, d), case["pool"], g)
    s["q"] = torch.randn((len(lens), R, hq, d), generator=g, device=DEV).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty(s["q"].shape, dtype=DTYPE[case["out_type"]], device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ passes
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _turn(x, cos, sin, paired):
    """x [tokens, heads, d] in 32 bits, its first elements turned by cos and sin [tokens, turned / 2]."""
    half = cos.shape[1]
    c, n = cos[:, None], sin[:, None]
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if paired else (x[..., :half], x[..., half:2 * half])
    u, v = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if paired else (y[..., :half], y[..., half:2 * half])
    u.copy_(a * c - b * n)
    v.copy_(b * c + a * n)
    return y


def _plain_rotate(s):
    c = s["case"]
    P, dtype = c["page"], DTYPE[c["pool"]]
    at, slot = s["positions"].long(), s["slots"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    q = _turn(s["q"].float(), cos, sin, c["paired"])
    k = _turn(s["new_k"].float(), cos, sin, c["paired"])
    for w, x in (("k", k), ("v", s["new_v"].float())):
        pool, x = s[w + "_pool"], x / s[w + "_scale"]
        if c["pool"] == "e4m3":
            pool.view(torch.uint8)[slot // P, :, slot % P] = x.clamp(-448, 448).to(dtype).view(torch.uint8)
        else:
            pool[slot // P, :, slot % P] = x.to(dtype)
    return {"q": q.to(s["q"].dtype), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_prompt(s):
    c = s["case"]
    h, hq, d, L = c["h_kv"], c["h_q"], c["d"], s["longest"]
    start = s["start"].long()
    B, G = start.numel() - 1, hq // h
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1
    i = t - start[b]

    def padded(x):
        y = torch.zeros((B, L, x.shape[1], d), device=DEV)
        y[b, i] = x.float()
        return y

    q = padded(s["q"]).view(B, L, h, G, d).permute(0, 2, 3, 1, 4).reshape(B, h, G * L, d)
    k, v = padded(s["k"]).permute(0, 2, 3, 1), padded(s["v"]).permute(0, 2, 1, 3)
    z = torch.matmul(q, k).mul_(s["scale"]).view(B, h, G, L, L)
    j = torch.arange(L, device=DEV)
    z.masked_fill_(j[None, :] > j[:, None], -math.inf)
    z.sub_(z.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(z.view(B, h, G * L, L), v).view(B, h, G, L, d) / z.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).reshape(B, L, hq, d)[b, i].to(torch.bfloat16)


def _read(s, w):
    """Keys or values as fp32 [batch, h, positions, d], through the block table."""
    ids = s["table"].clamp(min=0).long()
    pool = s[w + "_pool"]
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float().mul_(s[w + "_scale"])
    else:
        x = pool[ids].float()
    B, n, h, P, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, h, n * P, d)


def _plain_shared(s):
    c = s["case"]
    k, v = _read(s, "k"), _read(s, "v")
    B, R, hq, d = s["q"].shape
    h, L = k.shape[1], k.shape[2]
    G = hq // h
    q = s["q"].float().view(B, R, h, G, d).permute(0, 2, 3, 1, 4).reshape(B, h, G * R, d)
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, h, G, R, L)
    del k
    n = s["lens"].long()[:, None]
    p = n - R + torch.arange(R, device=DEV)[None, :]
    j = torch.arange(L, device=DEV)
    z.masked_fill_((j > p[:, :, None])[:, None, None], -math.inf)
    z.sub_(z.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(z.view(B, h, G * R, L), v).view(B, h, G, R, d) / z.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).reshape(B, R, hq, d).to(DTYPE[c["out_type"]])


def _own_rotate(s):
    import paged_split_kv_append_gb300 as nbx
    q = nbx.nbx_paged_kv_append_rotated(s["q"], s["new_k"], s["new_v"], s["cos"], s["sin"], s["positions"], s["k_pool"],
                                        s["v_pool"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                        interleaved=s["case"]["paired"], q_out=s["q_out"])
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_prompt(s):
    import paged_split_kv_append_gb300 as nbx
    return nbx.nbx_prompt_attn(s["q"], s["k"], s["v"], s["start"], s["scale"], out=s["out"])


def _own_shared(s):
    import paged_split_kv_append_gb300 as nbx
    if "workspace" not in s:   # what a serving loop keeps from step to step
        c = s["case"]
        size = nbx.nbx_paged_decode_shared_workspace_bytes(*s["q"].shape[:3], c["h_kv"], c["d"], s["max_len"],
                                                           s["shared"].numel())
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return nbx.nbx_paged_decode_attn_shared(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["max_len"],
                                            s["start"], s["shared"], s["scale"], k_scale=s["k_scale"],
                                            v_scale=s["v_scale"], out=s["out"], workspace=s["workspace"])


_run_plain = {"rotate": _plain_rotate, "prompt": _plain_prompt, "shared": _plain_shared}
_run_own = {"rotate": _own_rotate, "prompt": _own_prompt, "shared": _own_shared}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    return {"rotate": _exact_rotate, "prompt": _exact_prompt, "shared": _exact_shared}[case["op"]](prepare(case, seed))


def _exact_rotate(s):
    c = s["case"]
    half = c["turned"] // 2
    at, slot = s["positions"].long(), s["slots"].long()
    w = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]      # a turn is a product

    def turned(x):
        x = x.double()
        head, rest = x[..., :2 * half], x[..., 2 * half:]
        pairs = head.reshape(*head.shape[:-1], half, 2) if c["paired"] else \
            head.reshape(*head.shape[:-1], 2, half).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        y = y if c["paired"] else y.transpose(-1, -2)
        return torch.cat([y.reshape(head.shape), rest], -1)

    got = {"q": turned(s["q"])}
    for name, x in (("k", turned(s["new_k"])), ("v", s["new_v"].double())):
        pool = s[name + "_pool"].double()
        x = x / s[name + "_scale"]
        pool[slot // c["page"], :, slot % c["page"]] = x.clamp(-448, 448) if c["pool"] == "e4m3" else x
        got[name + "_pool"] = pool
    return got


def _exact_prompt(s):
    c = s["case"]
    G = c["h_q"] // c["h_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    start = s["start"].tolist()
    step = 2048
    for a, b in zip(start[:-1], start[1:]):
        for i in range(c["h_q"]):
            q = s["q"][a:b, i].double()
            k, v = s["k"][a:b, i // G].double(), s["v"][a:b, i // G].double()
            for lo in range(0, b - a, step):          # a block of rows, and the keys up to its last one
                hi = min(b - a, lo + step)
                z = (q[lo:hi] @ k[:hi].T) * s["scale"]
                z += torch.full_like(z, -math.inf).triu(lo + 1)
                out[a + lo:a + hi, i] = torch.softmax(z, -1) @ v[:hi]
    return out


def _exact_shared(s):
    c = s["case"]
    B, R, hq, d = s["q"].shape
    h, P = c["h_kv"], c["page"]
    out = torch.zeros((B, R, hq, d), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, : _ceil(n, P)].long()
        last = n - R + torch.arange(R, device=DEV)
        dark = torch.arange(n, device=DEV) > last[:, None]
        for i in range(h):
            kv = []
            for w in "kv":
                pool = s[w + "_pool"]
                x = pool.view(torch.uint8)[ids, i].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[ids, i]
                kv.append(x.double().reshape(-1, d)[:n] * s[w + "_scale"])
            heads = slice(i * (hq // h), (i + 1) * (hq // h))
            z = torch.einsum("rgd,jd->rgj", s["q"][b, :, heads].double(), kv[0]) * s["scale"]
            a = torch.softmax(z.masked_fill(dark[:, None], -math.inf), -1)
            out[b, :, heads] = torch.einsum("rgj,jd->rgd", a, kv[1])
    return out
