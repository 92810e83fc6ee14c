"""A serving loop's run through a session: prompts turned by their positions and appended, attended, forked into samples,
and the samples decoded step by step behind what they share. Against the same in 64 bits, on dense keys and values.

The cache holds what the append leaves (its own tests hold it to its roundings), so the decodes are compared with attention
over the pools' values; prompts with attention over the turned queries and keys as the call returns them. Tolerances are
those of tests/test_gpu_prompt.py and tests/test_gpu_shared.py."""

import math

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from paged_split_kv_append_gb300.session import PagedDecodeSession
from test_gpu_prompt import expect as expect_prompt, near as near_prompt
from test_gpu_rotated import near as near_rotated, turn
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LENS, SAMPLES, STEPS = [530, 300, 17], 3, 4     # the last prompt shares too little to be read apart


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


class Seen(Case):
    """What test_gpu_shared compares with, over a session's state."""

    def __init__(self, s, q):
        self.rows, self.h_q, self.h_kv, self.d, self.page = 1, s.h_q, s.h_kv, s.d, s.page_tokens
        self.lens_list, self.table, self.q, self.scale, self.out = s.seq_lens.tolist(), s.block_table, q, s.scale, s.out.dtype
        self.pools = [x.view(torch.float8_e4m3fn) if x.dtype is torch.uint8 else x for x in (s.k_pool, s.v_pool)]
        self.scales = [s.k_scale, s.v_scale]


@pytest.mark.parametrize("pool,out", [("bf16", torch.float32), ("bf16", torch.bfloat16), ("e4m3", torch.bfloat16)])
@pytest.mark.parametrize("d,h_q,h_kv,page", [(128, 8, 2, 16), (64, 6, 2, 64), (256, 12, 2, 32)])
def test_prompts_samples_and_steps(pool, out, d, h_q, h_kv, page):
    g = torch.Generator(device=DEV).manual_seed(d)
    batch, most = len(LENS) * (1 + SAMPLES), max(LENS) + STEPS + 1
    width = -(-most // page)
    num_pages = sum(-(-n // page) for n in LENS) + batch * 3
    s = PagedDecodeSession(num_pages=num_pages, h_kv=h_kv, page_tokens=page, d=d, pool_dtype=pool, batch=batch, rows=1,
                           h_q=h_q, max_seq_len=most, device=DEV, out_dtype=out, shared_groups=4)
    scale = 0.02 if pool == "e4m3" else 1.0
    # ---- the prompts, packed
    n = sum(LENS)
    table = torch.full((batch, width), -1, dtype=torch.int32)
    ids, at, rows = torch.randperm(num_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32), 0, []
    for i, m in enumerate(LENS):
        rows.append(i * (1 + SAMPLES))
        table[rows[-1], : -(-m // page)] = ids[at:at + -(-m // page)]
        at += -(-m // page)
    lens = [0] * batch
    for r, m in zip(rows, LENS):
        lens[r] = m
    s.set_inputs(torch.zeros((batch, 1, h_q, d), dtype=torch.bfloat16), table, lens, None, None, None, 1 / math.sqrt(d),
                 scale, scale)
    x = torch.randn((n, h_q + 2 * h_kv, d), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    angle = torch.arange(most, device=DEV, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(d // 2, device=DEV, dtype=torch.float64) / (d // 2))
    cos, sin = angle.cos().float(), angle.sin().float()
    positions = torch.cat([torch.arange(m) for m in LENS]).to(torch.int32).to(DEV)
    row_of = torch.cat([torch.full((m,), r) for r, m in zip(rows, LENS)]).to(DEV)

    def slots(row, pos):
        return (s.block_table[row, pos.long() // page] * page + pos % page).to(torch.int32)

    starts = ints([sum(LENS[:i]) for i in range(len(LENS) + 1)])
    raw_q, raw_k = q.clone(), k.clone()
    turned = s.append_rotated(q, k, v, cos, sin, positions, slots(row_of, positions), k_out=k)
    near_rotated(turned, *turn(raw_q, cos, sin, positions, False), 1)
    near_rotated(k, *turn(raw_k, cos, sin, positions, False), 1)
    o = s.prompt(turned, k, v, starts)
    for a, b in zip(starts.tolist()[:-1], starts.tolist()[1:]):
        near_prompt(o[a:b], *expect_prompt(turned, k, v, a, b, s.scale))
    # ---- each forked into samples
    src = ints([r for r in rows for _ in range(SAMPLES)])
    dst = ints([r + 1 + j for r in rows for j in range(SAMPLES)])
    s.fork(src, dst)
    s.set_groups(ints([r for r in rows] + [batch]), ints([m // page * page for m in LENS]))
    # ---- steps: a token for each, from a fresh page where the last is full
    free = [i for i in range(num_pages) if i not in set(s.block_table.flatten().tolist())]
    for _ in range(STEPS):
        held = s.seq_lens.tolist()
        for b in range(batch):
            if held[b] % page == 0:
                s.block_table[b, held[b] // page] = free.pop()
        x = torch.randn((batch, h_q + 2 * h_kv, d), generator=g, device=DEV).to(torch.bfloat16)
        at = s.seq_lens.clone()
        where = slots(torch.arange(batch, device=DEV), at)
        q1 = s.append_rotated(x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], cos, sin, at, where)
        s.seq_lens += 1
        s.q.copy_(q1[:, None])
        Seen(s, s.q).check(s.decode())
    with_groups = s.out.clone()
    s.set_groups(None, None)
    Seen(s, s.q).check(s.decode())
    tol = 2.0 ** -6 if out is torch.bfloat16 else 1e-4
    assert float((with_groups.double() - s.out.double()).abs().max()) <= tol * float(s.out.double().abs().max())
    assert s.status_bits() == 0


def test_a_captured_step_with_groups():
    """append_rotated and the grouped decode in one graph, replayed for new tokens and lengths."""
    h_q, h_kv, d, page, batch = 8, 2, 128, 16, 4
    g = torch.Generator(device=DEV).manual_seed(5)
    width, shared = 20, 160
    s = PagedDecodeSession(num_pages=100, h_kv=h_kv, page_tokens=page, d=d, pool_dtype="bf16", batch=batch, rows=1, h_q=h_q,
                           max_seq_len=width * page, device=DEV, fill_nan=False, shared_groups=1)
    s.k_pool.normal_(generator=g)
    s.v_pool.normal_(generator=g)
    table = torch.arange(batch * width, dtype=torch.int32).view(batch, width)
    table[:, : shared // page] = table[0, : shared // page]
    s.set_inputs(torch.zeros((batch, 1, h_q, d), dtype=torch.bfloat16), table, [161, 200, 250, 300], None, None, None, 0.1)
    s.set_groups(ints([0, batch]), ints([shared]))
    cos, sin = torch.rand((400, 64), generator=g, device=DEV), torch.rand((400, 64), generator=g, device=DEV)
    x = torch.randn((batch, h_q + 2 * h_kv, d), generator=g, device=DEV).to(torch.bfloat16)
    at, where = s.seq_lens - 1, torch.zeros(batch, dtype=torch.int32, device=DEV)
    rows = torch.arange(batch, device=DEV)

    def place():
        at.copy_(s.seq_lens - 1)
        where.copy_(s.block_table[rows, at.long() // page] * page + at % page)

    def step():
        s.append_rotated(x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], cos, sin, at, where, q_out=s.q.view(batch, h_q, d))
        return s.decode()

    place()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        s.seq_lens.copy_(ints([161 + 3 * i, 201 + i, 256 + i, 310]))
        x.copy_(torch.randn(x.shape, generator=g, device=DEV).to(torch.bfloat16))
        place()
        graph.replay()
        Seen(s, s.q).check(s.out)
    assert s.status_bits() == 0
