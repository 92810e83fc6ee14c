"""The cache operators together, as a serving loop uses them on one session: a prompt appended in chunks to a
block-scaled cache and attended with a cap and a window, forked into samples, stepped token by token, two rows
dropped, the pages compacted, and stepped on. After every move the outputs are compared with the definition
(oracle.cache) over caches kept on the host. Tolerances: tests/test_gpu_modified.py.
"""

import math

import numpy as np
import pytest
import torch

import oracle.cache as oc
import paged_split_kv_append_gb300 as nbx
from paged_split_kv_append_gb300.session import PagedDecodeSession

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGES, WIDTH, H_Q, H_KV, CAP, SPAN, PROMPTS, SAMPLES = 160, 16, 8, 2, 8.0, 50, (45, 130), 3


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


class Loop:
    """A session, and the same cache on the host."""

    def __init__(self, d, T, P, dtype):
        self.d, self.T, self.P, self.dtype = d, T, P, dtype
        self.B, self.scale = len(PROMPTS) * (1 + SAMPLES), 1.0 / math.sqrt(d)
        self.g = torch.Generator().manual_seed(d + T)
        self.s = s = PagedDecodeSession(num_pages=PAGES, h_kv=H_KV, page_tokens=P, d=d, pool_dtype="e4m3",
                                        batch=self.B, rows=1, h_q=H_Q, max_seq_len=256, device=DEV, scale_tokens=T)
        ids = np.random.default_rng(d).permutation(PAGES)
        self.table = np.full((self.B, WIDTH), -1, dtype=np.int32)
        for b, n in enumerate(PROMPTS):
            k = -(-n // P)
            self.table[b, :k] = ids[16 * b:16 * b + k]
        self.lens = np.zeros(self.B, dtype=np.int32)
        s.set_inputs(torch.zeros((self.B, 1, H_Q, d), dtype=torch.bfloat16), self.table, self.lens, None, None, None,
                     self.scale)
        self.codes = [t.cpu().numpy() for t in (s.k_pool, s.v_pool)]
        self.scales = [t.cpu().numpy() for t in (s.k_scales, s.v_scales)]

    def put(self):
        self.s.block_table.copy_(dev(self.table))
        self.s.seq_lens.copy_(dev(self.lens))

    def append(self, new):
        """new[b] tokens to every row: the step's inputs on the session, the append itself on the host's copy."""
        start = np.concatenate([[0], np.cumsum(new)])
        x = [(torch.randn((int(start[-1]), H_KV, self.d), generator=self.g) * (1 + 2 * w)).to(self.dtype)
             for w in range(2)]
        self.s.set_new_tokens(*x, self.lens, start)
        for w in range(2):
            oc.append_block_scaled(self.codes[w], self.scales[w], x[w].float().numpy(), self.table, self.lens, start,
                                   self.T)
        self.lens = (self.lens + np.asarray(new)).astype(np.int32)
        self.s.seq_lens.copy_(dev(self.lens))

    def query(self):
        self.s.q.copy_(torch.randn(self.s.q.shape, generator=self.g))
        self.begin = np.maximum(0, self.lens - SPAN)[:, None]
        self.s.set_modifications(softcap=CAP, key_begin=dev(self.begin))

    def move(self, moves):
        for src, dst, n in moves:
            for c, sc in zip(self.codes, self.scales):
                c[dst, :, :n] = c[src, :, :n]
                sc[dst, :, :-(-n // self.T)] = sc[src, :, :-(-n // self.T)]

    def check(self):
        s = self.s
        assert s.status_bits() == 0
        assert np.array_equal(s.block_table.cpu().numpy(), self.table)
        assert np.array_equal(s.seq_lens.cpu().numpy(), self.lens)
        values = [oc.pool_values(c, "e4m3", scales=x) for c, x in zip(self.codes, self.scales)]
        q = s.q.float().cpu().numpy()
        ref = oc.attention(q, *values, self.table, self.lens, self.scale, softcap=CAP, key_begin=self.begin)
        k, v = ([x[p, :, :min(self.P, n - j * self.P)] for n, row in zip(self.lens, self.table)
                 for j, p in enumerate(row) if j * self.P < n] for x in values)
        z = self.scale * np.linalg.norm(q, axis=-1).max() * max(np.linalg.norm(x, axis=-1).max() for x in k)
        tol = max(np.abs(x).max() for x in v) * (2.0 ** -19 * z + 2.0 ** -14)
        assert np.abs(s.out.double().cpu().numpy() - ref).max() <= tol

    def grant(self):
        """A page to every row that holds something and grows into a new one."""
        free = iter(sorted(set(range(PAGES)) - oc.pages_in_use(self.table, PAGES)))
        for b in np.nonzero((self.lens > 0) & (self.lens % self.P == 0))[0]:
            self.table[b, self.lens[b] // self.P] = next(free)
        self.put()

    def steps(self, n):
        """Tokens one by one to the rows that hold any."""
        for _ in range(n):
            self.grant()
            self.append((self.lens > 0).astype(np.int64))
            self.query()
            self.s.step()
            self.check()


@pytest.mark.parametrize("d,T,P,dtype", [(128, 16, 16, torch.bfloat16), (64, 32, 64, torch.float32)])
def test_a_serving_loop(d, T, P, dtype):
    c = Loop(d, T, P, dtype)
    for part in (0.4, 0.6):                       # the prompts, in two chunks that end inside blocks
        c.append([int(round(n * part)) for n in PROMPTS] + [0] * (c.B - len(PROMPTS)))
        c.query()
        c.s.step()
        c.check()
    src = np.repeat(np.arange(len(PROMPTS)), SAMPLES)
    dst = np.arange(len(PROMPTS), c.B)
    c.s.fork(dev(src), dev(dst))
    c.table, c.lens, moves = oc.fork(c.table, c.lens, src, dst, P, PAGES)
    c.move(moves)
    c.query()
    c.s.decode()
    c.check()
    c.steps(20)
    for b in (1, 4):                              # a prompt's own row and a sample are dropped
        c.table[b], c.lens[b] = -1, 0
    c.put()
    moves, counts = c.s.compact()
    c.table, want, live = oc.compact(c.table, c.lens, P, PAGES)
    c.move(want)
    assert counts.tolist() == [len(want), live] and [tuple(m) for m in moves[:len(want)].tolist()] == want
    c.steps(3)


def test_graphs_that_share_a_session():
    """A step, a fork and a compaction, captured one graph each over the same buffers and workspaces, replayed in
    turn."""
    c = Loop(128, 16, 16, torch.bfloat16)
    s = c.s
    c.append(list(PROMPTS) + [0] * (c.B - len(PROMPTS)))
    c.query()
    s.step()
    c.check()
    src, dst = np.array([0, 1, 1]), np.array([2, 3, 0])
    args = dev(src), dev(dst)
    keep = s.block_table, s.seq_lens, s.k_pool, s.v_pool, s.k_scales, s.v_scales
    was = [t.clone() for t in keep]
    room = torch.zeros((c.B, H_KV, c.d))          # a step's tokens: at most one a row, the rows behind them unread
    s.set_new_tokens(room.to(c.dtype), room.to(c.dtype), c.lens, np.zeros(c.B + 1))
    fixed = s.new_k, s.new_v, s.held, s.tok_start
    begin = torch.zeros((c.B, 1), dtype=torch.int32, device=DEV)
    s.set_modifications(softcap=CAP, key_begin=begin)
    graphs = []
    for call in (s.step, lambda: s.fork(*args), s.compact):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    step, fork, compact = graphs
    for t, x in zip(keep, was):
        t.copy_(x)
    for _ in range(2):
        fork.replay()
        c.table, c.lens, moves = oc.fork(c.table, c.lens, src, dst, c.P, PAGES)
        c.move(moves)
        compact.replay()
        c.table, moves, _ = oc.compact(c.table, c.lens, c.P, PAGES)
        c.move(moves)
        for _ in range(18):
            c.grant()
            c.append((c.lens > 0).astype(np.int64))
            for t, x in zip(fixed, (s.new_k, s.new_v, s.held, s.tok_start)):
                t[:x.shape[0]].copy_(x)
            c.query()
            begin.copy_(dev(c.begin))
            step.replay()
        c.check()
