"""The block-scaled append against its definition (oracle.cache), bit for bit.

Both sides do the same exactly rounded steps (a power-of-two scale, one rounding to E4M3), so codes and
scales have to be equal; positions that the call does not touch keep their bits.
"""

import numpy as np
import pytest
import torch

import oracle.cache as oc
import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


class Cache:
    """A block-scaled cache with random codes and power-of-two scales, on both sides."""

    def __init__(self, num_pages, h, P, d, T, seed):
        g = np.random.default_rng(seed)
        self.shape, self.T, self.P = (num_pages, h, P, d), T, P
        self.codes = [g.integers(0, 256, self.shape, dtype=np.uint8) for _ in range(2)]
        self.scales = [np.exp2(g.integers(-6, 3, (num_pages, h, P // T))).astype(np.float32) for _ in range(2)]
        self.dev = [torch.from_numpy(c.copy()).to(DEV) for c in self.codes]
        self.dev_scales = [torch.from_numpy(s.copy()).to(DEV) for s in self.scales]

    def append(self, new, table, lens, start, stream=None, status=None):
        dt = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)   # noqa: E731
        nbx.nbx_paged_kv_append_block_scaled(new[0], new[1], *self.dev, *self.dev_scales, dt(table), dt(lens),
                                             dt(start), status=status, stream=stream)
        for w in range(2):
            oc.append_block_scaled(self.codes[w], self.scales[w], new[w].float().cpu().numpy(), table, lens, start,
                                   self.T)

    def check(self):
        torch.cuda.synchronize()
        for w in range(2):
            assert np.array_equal(self.dev_scales[w].cpu().numpy(), self.scales[w])
            got, want = self.dev[w].cpu().numpy(), self.codes[w]
            nan = (got & 0x7F) == 0x7F
            assert np.array_equal(nan, (want & 0x7F) == 0x7F)     # a NaN's sign is not defined
            assert np.array_equal(got[~nan], want[~nan])


def table_for(lens, P, seed, spare=3):
    g = np.random.default_rng(seed)
    width = max(1, max(-(-n // P) for n in lens))
    need = [-(-n // P) for n in lens]
    ids = g.permutation(sum(need) + spare).astype(np.int32)
    t = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = ids[at:at + k]
        at += k
    return t, sum(need) + spare


def new_tokens(n, h, d, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn((n, h, d), generator=g) * torch.exp(spread * torch.randn((n, h, 1), generator=g)))
            .to(dtype).to(DEV) for _ in range(2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,h,P,T", [(64, 1, 16, 16), (128, 3, 32, 16), (256, 2, 64, 64), (128, 8, 128, 128),
                                     (64, 5, 96, 32), (256, 1, 256, 128), (128, 2, 64, 32)])
def test_append_matches_the_definition(dtype, d, h, P, T):
    # no token, one, up to a block's end, across blocks and pages, from held lengths inside and on blocks
    lens = [0, 1, 15, 16, 17, 5, T - 1, T, T + 1, P - 1, P, 2 * P + 3, 0]
    new = [0, 1, 1, 1, 30, 11, 1, T, P, 2, 3 * P + 7, 1, 2 * T + 5]
    start = np.concatenate([[0], np.cumsum(new)])
    table, pages = table_for([a + n for a, n in zip(lens, new)], P, 1)
    c = Cache(pages, h, P, d, T, 2)
    c.append(new_tokens(int(start[-1]), h, d, dtype, 3), table, lens, start)
    c.check()


def test_one_token_at_a_time_rescales_held_codes():
    # 40 steps of growing magnitude: every step raises some block's scale over held codes
    lens, P, T, h, d = [3, 0, 31], 32, 16, 2, 128
    table, pages = table_for([n + 40 for n in lens], P, 4)
    c = Cache(pages, h, P, d, T, 5)
    for step in range(40):
        x = [t * 1.4 ** step for t in new_tokens(3, h, d, torch.float32, 10 + step, spread=1.0)]
        c.append(x, table, [n + step for n in lens], [0, 1, 2, 3])
    c.check()


def test_appending_again_changes_nothing():
    lens, P, T = [7, 20], 32, 16
    table, pages = table_for([40, 60], P, 6)
    c = Cache(pages, 2, P, 64, T, 7)
    x = new_tokens(73, 2, 64, torch.bfloat16, 8)
    c.append(x, table, lens, [0, 33, 73])
    c.check()
    before = [t.clone() for t in c.dev + c.dev_scales]
    c.append(x, table, lens, [0, 33, 73])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, c.dev + c.dev_scales))


def test_infinities_nan_zeros_and_the_ends_of_the_range():
    P, T, h, d = 16, 16, 1, 64
    rows = [np.zeros(d), np.full(d, 1e-30), np.full(d, 3e38), np.full(d, 448.0), np.full(d, np.nextafter(np.float32(448), np.float32(1e9))),
            np.full(d, 1e-42), np.full(d, 2.0 ** 57)]
    rows.append(np.where(np.arange(d) == 3, np.inf, 1.0))
    rows.append(np.where(np.arange(d) == 3, np.nan, 2.0))
    rows.append(np.where(np.arange(d) % 2 == 0, -np.inf, np.nan))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)[:, None, :]).to(DEV)
    n = len(rows)
    table, pages = table_for([1] * n, P, 9)
    c = Cache(pages, h, P, d, T, 10)
    with np.errstate(invalid="ignore", over="ignore"):
        c.append([x, -x], table, [0] * n, list(range(n + 1)))
    c.check()


def test_bad_sequences_are_skipped_with_their_bit_and_others_written():
    P, T, h, d = 16, 16, 2, 64
    lens = [0, 5, 0, 9]
    table, pages = table_for([20, 20, 20, 20], P, 11)
    good = table.copy()
    cases = [("page", nbx.DEV_BAD_PAGE), ("page_high", nbx.DEV_BAD_PAGE), ("len", nbx.DEV_BAD_LEN),
             ("past", nbx.DEV_BAD_LEN), ("start", nbx.DEV_BAD_LEN), ("scale", nbx.DEV_BAD_SCALE)]
    for what, bit in cases:
        c = Cache(pages, h, P, d, T, 12)
        x = new_tokens(40, h, d, torch.float32, 13)
        start, ln, tb = np.array([0, 10, 20, 30, 40]), np.array(lens), good.copy()
        if what == "page":
            tb[1, 0] = -1
        elif what == "page_high":
            tb[1, 0] = pages
        elif what == "len":
            ln[1] = -1
        elif what == "past":
            ln[1] = 2 * P
        elif what == "start":
            start = np.array([0, 10, 9, 30, 41])
        else:
            c.dev_scales[0][tb[1, 0]] = float("nan")
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        dt = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)   # noqa: E731
        nbx.nbx_paged_kv_append_block_scaled(x[0], x[1], *c.dev, *c.dev_scales, dt(tb), dt(ln), dt(start),
                                             status=status)
        torch.cuda.synchronize()
        assert int(status.item()) & bit, what
        # sequence 0 is written whatever the others are
        ref = Cache(pages, h, P, d, T, 12)
        oc.append_block_scaled(ref.codes[0], ref.scales[0], x[0].cpu().numpy(), good[:1], [0], [0, 10], T)
        pg = good[0, 0]
        assert np.array_equal(c.dev[0][pg, :, :10].cpu().numpy(), ref.codes[0][pg, :, :10]), what


def test_many_sequences_and_a_second_stream():
    # more sequences than one 32-way step of the search tells apart, on a side stream
    B, P, T, h, d = 1500, 16, 16, 1, 64
    g = np.random.default_rng(14)
    lens, new = g.integers(0, 20, B), g.integers(0, 4, B)
    start = np.concatenate([[0], np.cumsum(new)])
    table, pages = table_for(list(lens + new), P, 15)
    c = Cache(pages, h, P, d, T, 16)
    x = new_tokens(int(start[-1]), h, d, torch.bfloat16, 17)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.append(x, table, lens, start)
    s.synchronize()
    c.check()
