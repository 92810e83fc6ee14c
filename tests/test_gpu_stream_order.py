"""Calls in stream order may reuse one another's memory, and a plan that starts while the grid ahead of it still
runs may not be seen to: decodes back to back on one workspace, and decodes whose workspace lies where the call
before them still reads. Every result has to equal, bit for bit, that of the same call alone."""

import numpy as np
import pytest
import torch

import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OTHER = 4     # sequences of the smaller call


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    nbx.nbx_set_decode_grid_limit(0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Cache:
    def __init__(self, batch, longest, pool=torch.float32, h_kv=8, h_q=32, d=128, P=16, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        lens = np.random.default_rng(seed).integers(1, longest + 1, batch)
        lens[0] = longest
        width = -(-longest // P)
        self.longest, self.lens = longest, dev(lens)
        self.table = dev(np.random.default_rng(seed).permutation(batch * width).reshape(batch, width))
        shape = (batch * width, h_kv, P, d)
        self.k, self.v = (torch.randn(shape, generator=g, device=DEV).to(pool) for _ in range(2))
        self.q = torch.randn((batch, 1, h_q, d), generator=g, device=DEV)
        if pool != torch.float32:
            self.q = self.q.to(torch.bfloat16)
        self.out = torch.empty(self.q.shape, device=DEV)

    def args(self):
        return self.q, self.k, self.v, self.table, self.lens, self.longest, 0.088

    def plain(self, ws):
        return nbx.nbx_paged_decode_attn(*self.args(), out=self.out, workspace=ws)

    def modified(self, ws):
        return nbx.nbx_paged_decode_attn_modified(*self.args(), softcap=5.0, out=self.out, workspace=ws)


@pytest.mark.parametrize("first,pool,longest", [("plain", torch.float32, 256), ("modified", torch.float32, 512),
                                                ("plain", torch.bfloat16, 256), ("modified", torch.bfloat16, 127)])
def test_decodes_back_to_back_on_one_workspace(first, pool, longest):
    # the first has one split a sequence, so no merge stands between it and the second's plan, and several times as
    # many work units as a grid takes at once; the second is a smaller call with a list of its own
    a, b = Cache(600, longest, pool, seed=1), Cache(OTHER, longest, pool, seed=2)
    need = max(nbx.nbx_paged_decode_modified_workspace_bytes(600, 1, 32, 8, 128, longest), 256)
    ws, apart = (torch.zeros(need, dtype=torch.uint8, device=DEV) for _ in range(2))
    want = []
    for c, kind in ((a, first), (b, "plain"), (a, "plain")):
        want.append(getattr(c, kind)(apart).clone())
        torch.cuda.synchronize()
    outs = [torch.empty_like(w) for w in want]

    def run():
        for c, kind, o in ((a, first, outs[0]), (b, "plain", outs[1]), (a, "plain", outs[2])):
            c.out = o
            getattr(c, kind)(ws)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        for replay in (graph.replay, run):
            for o in outs:
                o.fill_(float("nan"))
            replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_workspace_where_the_append_ahead_reads_its_tokens():
    c = Cache(OTHER, 256, torch.bfloat16, seed=3)
    n = 20000
    g = torch.Generator(device=DEV).manual_seed(4)
    need = nbx.nbx_paged_decode_workspace_bytes(OTHER, 1, 32, 8, 128, 256)
    room = torch.empty(2 * n * 8 * 128 * 2, dtype=torch.uint8, device=DEV)
    new_k, new_v = room.view(torch.bfloat16).view(2, n, 8, 128)
    assert need <= room.numel()
    ws = room[:need]                       # over the first tokens of new_k
    x = torch.randn((2, n, 8, 128), generator=g, device=DEV).to(torch.bfloat16)
    pool = [torch.zeros((n // 16, 8, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    slots = dev(np.random.default_rng(5).permutation(n))
    codes = [torch.zeros((n // 16, 8, 16, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones((n // 16, 8, 1), device=DEV) for _ in range(2)]
    table, zero, start = dev(np.arange(n // 16)[None]), dev([0]), dev([0, n])
    alone = c.plain(torch.empty(need, dtype=torch.uint8, device=DEV)).clone()

    def appended(ws):
        new_k.copy_(x[0])
        new_v.copy_(x[1])
        nbx.nbx_paged_kv_append(new_k, new_v, *pool, slots)
        if ws is not None:
            c.plain(ws)
        new_k.copy_(x[0])
        nbx.nbx_paged_kv_append_block_scaled(new_k, new_v, *codes, *scales, table, zero, start)
        if ws is not None:
            c.plain(ws)
        torch.cuda.synchronize()
        return [t.clone() for t in pool + codes + scales]

    want = appended(None)
    for _ in range(5):
        got = appended(ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(c.out, alone)


def test_a_workspace_where_the_copies_ahead_read_their_moves():
    # a fork, a compaction and a copy, each followed by a decode whose workspace holds the list of moves
    c = Cache(OTHER, 256, torch.bfloat16, seed=6)
    need = nbx.nbx_paged_decode_workspace_bytes(OTHER, 1, 32, 8, 128, 256)
    alone = c.plain(torch.empty(need, dtype=torch.uint8, device=DEV)).clone()
    pages, n = 4000, 1000
    room = torch.empty(max(need, 256 + 3 * 4 * pages), dtype=torch.uint8, device=DEV)
    moves = room[256:256 + 12 * n].view(torch.int32).view(n, 3)
    count = room[:4].view(torch.int32)
    pair = torch.stack([torch.arange(n), torch.arange(n) + 2000, torch.full((n,), 16)], 1).int().to(DEV)
    pool = [torch.randn((pages, 4, 16, 128), device=DEV).to(torch.bfloat16) for _ in range(2)]
    for _ in range(5):
        for t in pool:
            t[2000:].zero_()
        moves.copy_(pair)
        count.fill_(n)
        nbx.nbx_paged_kv_copy_pages(moves, count, *pool)
        c.plain(room[:need])
        torch.cuda.synchronize()
        assert all(torch.equal(t[2000:2000 + n], t[:n]) and not bool(t[3000:].any()) for t in pool)
        assert torch.equal(c.out, alone)
        lens, table = dev([16 * 100 + 5] * n + [0] * n), torch.full((2 * n, 101), -1, dtype=torch.int32, device=DEV)
        table[:n] = torch.arange(n, device=DEV)[:, None].int()      # a row's pages are one page over and over
        ws = torch.empty(nbx.nbx_paged_kv_fork_workspace_bytes(2 * n, 101, n, pages), dtype=torch.uint8, device=DEV)
        nbx.nbx_paged_kv_fork(table, lens, dev(np.arange(n)), dev(np.arange(n) + n), *pool, moves=moves, n_moves=count,
                              workspace=ws)
        c.plain(room[:need])
        torch.cuda.synchronize()
        assert table[n:, 100].tolist() == list(range(n, 2 * n)) and torch.equal(c.out, alone)
        assert all(torch.equal(t[n:2 * n, :, :5], t[:n, :, :5]) for t in pool)
