"""The shared-prefix decode against its definition in 64 bits, which knows of no groups.

Tolerance of an output o = sum a_j v_j, with M = sum a_j |v_j| (a: the exact weights):
- a score's fp32 sum of d exact products is off by at most d 2^-23 S, S = scale sum |q_i k_i|, its factor and the
  difference to the maximum by 2^-23 of the largest |z| each, exp2 by 2^-21: E = d 2^-23 S + 2^-22 max |z| + 2^-21 of a
  weight, numerator and denominator: 2 E M. Sums over n keys and the merge add (n + 64) 2^-23 M.
- fp32 output: prefix weights are three bf16 terms, each rounding what the one before left by half a step, 2^-24 M, or two
  f16 ones, 2^-22 M and 2^-25 of a weight of 2^7 or more in the sum for each of n keys: 2^-32 n max |v|. The own positions'
  weights are as exact as fp32.
- bf16 output: prefix weights rounded to bf16, 2^-8 M, their splits' results too, 2^-8 M; the output's own rounding 2^-8 |o|.
E4M3 pools: their values are what the codes stand for, exactly; queries as f16 after a power of two are exact but for
elements under 2^-24 of the vector's largest (2^-25 of it each: d 2^-25 max|q| max|k| scale more in E); weights as f16 terms
are better than bf16 ones.
"""

import math

import pytest
import torch

import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """groups: a list of (shared positions, lengths of the members)."""

    def __init__(self, groups, rows, h_q, h_kv, d, page, pool="bf16", out="f32", seed=0, q_type="bf16", spare=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens_list = [n for _, m in groups for n in m]
        self.starts_list = [0]
        for _, m in groups:
            self.starts_list.append(self.starts_list[-1] + len(m))
        self.rows, self.h_q, self.h_kv, self.d, self.page = rows, h_q, h_kv, d, page
        need = sum(a // page + sum(max(0, -(-n // page) - a // page) for n in m) for a, m in groups)
        self.num_pages = need + spare
        ids = torch.randperm(self.num_pages, generator=g, device=DEV).to(torch.int32)
        width = max(1, max(-(-n // page) for n in self.lens_list))
        self.table = torch.full((len(self.lens_list), width), -1, dtype=torch.int32, device=DEV)
        at = b = 0
        for a, m in groups:
            common = ids[at:at + a // page]
            at += a // page
            for n in m:
                k = -(-n // page)
                s = min(a // page, k)
                self.table[b, :s] = common[:s]
                self.table[b, s:k] = ids[at:at + max(0, k - s)]
                at += max(0, k - s)
                b += 1
        self.lens, self.start, self.shared = ints(self.lens_list), ints(self.starts_list), ints([a for a, _ in groups])
        shape = (self.num_pages, h_kv, page, d)
        self.pools, self.scales = [], []
        for _ in range(2):
            x = torch.randn(shape, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))
            s = 1.0
            if pool == "e4m3":
                s = float(x.abs().max()) / 448.0
                x = (x / s).clamp(-448, 448)
            x = x.to(TYPES[pool])
            # the pages of no row, and the positions behind each sequence's last, hold NaN
            self.pools.append(x)
            self.scales.append(s)
        self.poison()
        self.q = torch.randn((len(self.lens_list), rows, h_q, d), generator=g, device=DEV).to(TYPES[q_type])
        self.scale = 1 / math.sqrt(d)
        self.out = TYPES[out]
        self.max_len = max(1, max(self.lens_list))

    def poison(self):
        held = torch.zeros((self.num_pages, self.page), dtype=torch.bool, device=DEV)
        for b, n in enumerate(self.lens_list):
            j = torch.arange(n, device=DEV)
            held[self.table[b, j // self.page].long(), j % self.page] = True
        for x in self.pools:
            raw = x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x
            raw[(~held)[:, None].expand(-1, self.h_kv, -1)] = 0x7F if raw.dtype is torch.uint8 else float("nan")

    def run(self, **kw):
        args = dict(k_scale=self.scales[0], v_scale=self.scales[1], out_dtype=self.out)
        args.update(kw)
        return nbx.nbx_paged_decode_attn_shared(self.q, *self.pools, self.table, self.lens, self.max_len, self.start,
                                                self.shared, self.scale, **args)

    def expect(self, b):
        n, R, G = self.lens_list[b], self.rows, self.h_q // self.h_kv
        ids = self.table[b, : -(-n // self.page)].long()
        kv = []
        for x, s in zip(self.pools, self.scales):
            y = x.view(torch.uint8)[ids].view(x.dtype) if x.dtype is torch.float8_e4m3fn else x[ids]
            kv.append(y.double().permute(1, 0, 2, 3).reshape(self.h_kv, -1, self.d)[:, :n] * s)
        q = self.q[b].double().view(R, self.h_kv, G, self.d)
        z = torch.einsum("rhgd,hjd->rhgj", q, kv[0]) * self.scale
        dark = (torch.arange(n, device=DEV) > (n - R + torch.arange(R, device=DEV))[:, None])[:, None, None]
        z = z.masked_fill(dark, -math.inf)
        a = torch.softmax(z, -1)
        a = torch.where(z.amax(-1, keepdim=True) == -math.inf, torch.zeros_like(a), a)
        o = torch.einsum("rhgj,hjd->rhgd", a, kv[1])
        M = torch.einsum("rhgj,hjd->rhgd", a, kv[1].abs())
        S = torch.einsum("rhgd,hjd->rhgj", q.abs(), kv[0].abs()) * abs(self.scale)
        big = z.masked_fill(dark, 0.0).abs().amax(-1, keepdim=True)
        E = self.d * 2.0 ** -23 * S.amax(-1, keepdim=True) + 2.0 ** -22 * big + 2.0 ** -21
        if self.pools[0].dtype is torch.float8_e4m3fn:
            E = E + self.d * 2.0 ** -25 * float(q.abs().max()) * float(kv[0].abs().max()) * abs(self.scale)
        tol = (2 * E + (n + 64) * 2.0 ** -23 + (2.0 ** -7 if self.out is torch.bfloat16 else 2.0 ** -22)) * M + \
            n * 2.0 ** -32 * float(kv[1].abs().max())
        if self.out is torch.bfloat16:
            tol = (tol + 2.0 ** -8 * o.abs()) * (1 + 2.0 ** -7)
        return o.reshape(R, self.h_q, self.d), tol.reshape(R, self.h_q, self.d)

    def check(self, out):
        torch.cuda.synchronize()
        assert out.dtype is self.out and out.shape == self.q.shape
        for b, n in enumerate(self.lens_list):
            got = out[b].double()
            if n == 0:
                assert bool((got == 0).all())
                continue
            want, tol = self.expect(b)
            off = (got - want).abs() - tol
            assert bool(torch.isfinite(got).all()) and float(off.max()) <= 0, (b, n, float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
def test_pages_types_and_widths(pool, out, d, page):
    n = 768
    Case([(n, [n + 5, n + 70, n + 1]), (n + 3 * page, [n + 4 * page, n + 7 * page + 3])], 1, 8, 2, d, page, pool, out,
         d + page).check_run()


def _check_run(self, **kw):
    status = ints([0])
    self.check(self.run(status=status, **kw))
    assert int(status) == 0


Case.check_run = _check_run


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (4, 4), (6, 1), (24, 4), (7, 1), (40, 2), (128, 1), (160, 1), (33, 3)])
@pytest.mark.parametrize("rows", [1, 3])
def test_heads_and_rows(out, h_q, h_kv, rows):
    Case([(640, [700, 650, 800, 643]), (256, [300, 260])], rows, h_q, h_kv, 128, 32, "bf16", out, h_q + rows).check_run()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("groups", [
    [(128, [129, 130])], [(112, [300, 301])], [(4096, [4097])], [(4096, [4096 + 31] * 40)], [(0, [5, 9, 1])],
    [(1024, [1025, 0, 1100, 0])], [(1024, [0, 0, 1100, 1030]), (512, [0, 0])], [(5000, [5010, 5011]), (0, [7]), (300, [310, 1300])],
    [(2000, [2001, 2000, 2064])], [(2048, [2048, 2049, 3000])], [(384, [390 + i for i in range(130)])]], ids=str)
def test_groups(pool, d, groups):
    Case(groups, 1, 8, 2, d, 16, pool, "f32", 3).check_run()


def test_many_sequences_and_groups():
    """More of both than the plan holds in shared memory, among them empty sequences and groups of one."""
    g = torch.Generator().manual_seed(11)
    groups = []
    for i in range(700):
        n = (128, 256, 0, 160)[i % 4]
        members = torch.randint(n, n + 90, (1 + i % 6,), generator=g).tolist()
        groups.append((n, [0 if i % 9 == 0 and j == 1 else max(1, m) for j, m in enumerate(members)]))
    c = Case(groups, 1, 2, 1, 64, 16, "bf16", "f32", 12)
    assert len(c.lens_list) > 2048
    c.check_run()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_pages_whose_offsets_pass_32_bits(pool):
    c = Case([(1024, [1100, 1500, 1030]), (512, [600, 513])], 1, 8, 8, 128, 256, pool, "f32", 13,
             spare=(1 << 32) // (8 * 256 * 128 * (2 if pool == "bf16" else 1)) + 3000)
    assert int(c.table.max()) * 8 * 256 * 128 * c.pools[0].element_size() > 1 << 32
    c.check_run()


def test_what_is_said_to_be_shared_is_cut_to_what_every_row_sees():
    """A prefix that runs into a member's own new rows, one that is no whole number of pages, one past a length."""
    c = Case([(1024, [1024, 1030, 1100]), (700, [760, 800])], 4, 8, 2, 128, 64, "bf16", "f32", 4)
    c.shared = ints([1 << 30, 743])      # the rows of the first group do hold the same pages up to 1024
    out = c.run()
    # 743 are 11 whole pages, of which the rows hold 10 in common: the last row is read as if it held the first's
    own = c.table.clone()
    c.table[4, :11] = c.table[3, :11]
    c.check(out)
    c.table = own
    c.shared = ints([1023, 1])
    c.check_run()


@pytest.mark.parametrize("start,shared", [([0, 3, 2], [512, 512]), ([-1, 2, 5], [512, 512]), ([0, 2, 6], [512, 512]),
                                          ([0, 3, 5], [-1, 512])])
def test_groups_that_make_no_sense(start, shared):
    c = Case([(512, [600, 700, 800]), (512, [520, 530])], 1, 4, 2, 64, 16, "bf16", "f32", 5)
    c.start, c.shared = ints(start), ints(shared)
    status = ints([0])
    c.check(c.run(status=status))
    assert int(status) == nbx.DEV_BAD_ROW


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_bad_page_in_the_prefix_and_a_bad_length(pool, d):
    c = Case([(1024, [1100, 1050, 1200])], 1, 8, 2, d, 16, pool, "f32", 6)
    for page in (-1, c.num_pages, 1 << 30):
        was = c.table.clone()
        c.table[:, 10] = page
        status = ints([0])
        out = c.run(status=status)
        assert int(status) == nbx.DEV_BAD_PAGE and bool(torch.isfinite(out).all())
        # the tile's positions are skipped: the result of the other positions
        c2 = Case([(1024, [1100, 1050, 1200])], 1, 8, 2, d, 16, pool, "f32", 6)
        keep = [i for i in range(c2.table.shape[1]) if i != 10]
        c2.table = c2.table[:, keep].contiguous()
        c2.lens_list = [n - 16 for n in c2.lens_list]
        c2.lens, c2.shared, c2.max_len = ints(c2.lens_list), ints([1008]), 1184
        c2.check(out)
        c.table = was
    c.lens = ints([1100, -1, 1 << 20])
    status = ints([0])
    out = c.run(status=status)
    assert int(status) == nbx.DEV_BAD_LEN
    assert bool((out[1:] == 0).all())
    c.lens_list = c.lens_list[:1]
    want, tol = c.expect(0)
    assert float(((out[0].double() - want).abs() - tol).max()) <= 0


# ---- sequences of 8 query vectors to a KV head and more, whose own positions the tiles read too
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("rows,h_q", [(4, 8), (1, 16), (20, 4)])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_own_positions_of_many_vectors(page, d, out, rows, h_q, pool):
    """Own positions of no, one and many tiles, sequences shorter than their rows, of no group, and empty."""
    groups = [(768, [769, 768 + 255, 768 + 256, 768 + 257, 1900]), (0, [1, 5, 0, 2000]), (0, [130]), (300, [300, 0, 431])]
    Case(groups, rows, h_q, 2, d, page, pool, out, page + d).check_run()


@pytest.mark.parametrize("n", [0, 3])
def test_many_sequences_of_many_vectors(n):
    g = torch.Generator().manual_seed(11 + n)
    groups = []
    for i in range(500):
        shared = (128, 0, 160)[i % 3]
        members = torch.randint(shared, shared + 90, (2 + i % 5 + n,), generator=g).tolist()
        groups.append((shared, [0 if i % 7 == 0 and j == 1 else max(1, m) for j, m in enumerate(members)]))
    c = Case(groups, 2, 4, 1, 64, 16, "bf16", "bf16", 12)
    assert (len(c.lens_list) > 2048) == (n == 3)
    c.check_run()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_scales_of_many_vectors(d, scale, pool):
    c = Case([(1024, [1100, 1030]), (0, [333])], 3, 8, 2, d, 16, pool, "f32", 8)
    c.scale = scale
    c.check_run()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_a_bad_page_among_own_positions_of_many_vectors(d, out, pool):
    for page in (-1, 1 << 30):
        c = Case([(1024, [1100, 1500])], 1, 16, 2, d, 16, pool, out, 14)
        c.table[1, 70] = page
        status = ints([0])
        out_t = c.run(status=status)
        torch.cuda.synchronize()
        assert int(status) == nbx.DEV_BAD_PAGE
        want, tol = c.expect(0)
        assert bool(((out_t[0].double() - want).abs() <= tol).all())
        c.table = c.table[:, [i for i in range(c.table.shape[1]) if i != 70]].contiguous()
        c.lens_list = [1100, 1500 - 16]
        want, tol = c.expect(1)
        assert bool(((out_t[1].double() - want).abs() <= tol).all())


def test_streams_and_graphs_of_many_vectors():
    a = Case([(512, [700, 620]), (0, [90])], 4, 8, 2, 128, 32, "bf16", "bf16", 15)
    b = Case([(640, [700, 900])], 4, 8, 2, 128, 32, "bf16", "bf16", 16)
    want = [a.run().clone(), b.run().clone()]
    outs = [torch.empty_like(w) for w in want]
    ws = nbx.nbx_paged_decode_shared_workspace_bytes(3, 4, 8, 2, 128, 900, 2)
    ws = torch.empty(ws, dtype=torch.uint8, device=DEV)
    graphs = []
    for c, o in zip((a, b), outs):   # two graphs over one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, c, o in zip(streams, (a, b), outs):
            o.zero_()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                c.run(out=o)
            torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("q_type,pool", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "e4m3")])
def test_formats_whose_groups_are_ignored(q_type, pool):
    c = Case([(512, [600, 700, 513])], 2, 4, 2, 64, 16, pool, "f32", 7, q_type=q_type)
    c.check_run()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    c = Case([(1024, [1100, 1030])], 1, 8, 2, 128, 16, "bf16", "f32", 8)
    c.scale = scale
    c.check_run()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_nan_in_the_prefix_reaches_all_of_its_head(pool, where):
    c = Case([(1024, [1100, 1030]), (256, [300, 301])], 1, 8, 2, 128, 16, pool, "f32", 9)
    x = c.pools[0 if where == "k" else 1]
    raw = x.view(torch.uint8) if pool == "e4m3" else x
    raw[int(c.table[0, 20]), 1, 3, 17] = 0x7F if pool == "e4m3" else float("nan")
    out = c.run()
    nan = torch.isnan(out)
    assert not bool(nan[:, :, :4].any()) and not bool(nan[2:].any())
    assert bool(nan[:2, :, 4:, 17].all())
    assert bool(nan[:2, :, 4:].all()) == (where == "k")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d,h_q,rows", [(64, 8, 4), (128, 8, 4), (256, 8, 4), (128, 4, 4), (128, 24, 40), (256, 6, 70)])
@pytest.mark.parametrize("pool,bad", [("bf16", float("nan")), ("bf16", float("inf")), ("e4m3", float("nan"))])
def test_values_of_later_rows_do_not_reach_earlier_ones(d, h_q, rows, out, pool, bad):
    """In a sequence's last positions, which its last rows alone see: at the last and at row r's own; in a split's first key
    tile, and in one whose maximum is an earlier tile's."""
    c = Case([(512, [700, 620]), (0, [rows, 300, 120])], rows, h_q, 2, d, 32, pool, out, 21)

    def put(kv, b, x, head, column, value):
        y = c.pools[kv]
        if pool == "e4m3":
            y, value = y.view(torch.uint8), 0x7F if value != 0 else 0
        y[c.table[b, x // 32].long(), head, x % 32, column] = value

    hit = {0: rows - 1, 3: rows // 2, 4: rows - 1}   # sequence -> the first row that sees the value
    at = {b: c.lens_list[b] - rows + r for b, r in hit.items()}
    for b, x in at.items():
        put(1, b, x, 1, 5, bad)
        put(0, b, x, 0, 7, bad)
    out = c.run()
    torch.cuda.synchronize()
    for b, x in at.items():
        r, h = hit[b], h_q // 2
        assert bool(torch.isfinite(out[b, :r]).all())
        assert not bool(torch.isfinite(out[b, r:, h:, 5]).any())
        # a NaN among the key's elements leaves no score; +inf a score of -inf to a vector that is negative there (the
        # scale is positive), which takes the key's weight away and leaves the others
        spared = (c.q[b, r:, :h, 7] < 0) & (bad == float("inf"))
        assert torch.equal(torch.isfinite(out[b, r:, :h]).all(-1), spared)
        put(1, b, x, 1, 5, 0)
        put(0, b, x, 0, 7, 0)
        want, tol = c.expect(b)
        assert bool(((out[b].double() - want).abs() <= tol)[:r].all())
    for b in (1, 2):
        want, tol = c.expect(b)
        assert bool(((out[b].double() - want).abs() <= tol).all())


def test_page_ids_do_not_matter_and_the_same_again():
    c = Case([(2048, [2100, 2060, 3000]), (512, [530, 700])], 2, 8, 2, 128, 16, "bf16", "f32", 10)
    one = c.run()
    assert torch.equal(one, c.run())
    perm = torch.randperm(c.num_pages, device=DEV)
    c.pools = [x[torch.argsort(perm)].contiguous() for x in c.pools]
    t = c.table.long()
    c.table = torch.where(t >= 0, perm[t.clamp(min=0)], t).to(torch.int32)
    assert torch.equal(one, c.run())


def test_another_stream_a_replayed_graph_and_two_calls_at_once():
    a = Case([(1024, [1100, 1030, 2000])], 1, 8, 2, 128, 16, "bf16", "bf16", 11)
    b = Case([(512, [700, 530]), (256, [300, 500])], 1, 8, 2, 128, 16, "bf16", "bf16", 12)
    torch.cuda.synchronize()
    sides, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        outs.append((a, b)[i % 2].run(stream=sides[i % 2]))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        (a, b)[i % 2].check(o)
    ws = torch.empty(nbx.nbx_paged_decode_shared_workspace_bytes(3, 1, 8, 2, 128, a.max_len, 1), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(outs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(out=out, workspace=ws, out_dtype=None)
    a.q.neg_()
    a.lens.copy_(ints([1090, 1025, 1500]))
    a.lens_list = [1090, 1025, 1500]
    a.shared.copy_(ints([800]))
    graph.replay()
    a.check(out)
    graph.replay()
    a.check(out)


def test_refusals_of_the_binding():
    c = Case([(512, [600, 700])], 1, 4, 2, 64, 16, "bf16", "f32", 13)
    with pytest.raises(ValueError):
        c.run(out=torch.empty_like(c.q), out_dtype=torch.float32)
    with pytest.raises(ValueError):
        c.run(status=ints([0])[1:])
    for name, bad in (("start", ints([0])), ("start", c.start.long()), ("shared", c.shared.float()), ("lens", ints([1])),
                      ("table", c.table[:1]), ("shared", c.shared.cpu()), ("q", c.q[:, :, :, :32].contiguous())):
        was = getattr(c, name)
        setattr(c, name, bad)
        with pytest.raises((ValueError, nbx.NbxError)):
            c.run()
        setattr(c, name, was)
    with pytest.raises(nbx.NbxError):
        c.run(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    c.start, c.shared = ints([0]), ints([])     # no groups: a plain decode
    c.check_run()
