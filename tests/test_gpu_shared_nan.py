"""NaN scores in the shared-prefix decode: a row that sees one gets NaN, whatever else lies in its splits, and no other row
does. Finite rows are held to the definition in 64 bits, with the tolerances of test_gpu_shared.py."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_shared import Case, ints

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# query vectors to a KV head: below 8 (own positions by the one-warp kernel) and from 8 on (in the tiles)
VECTORS = [(1, 4, 2), (1, 16, 2), (3, 8, 2)]
# members without positions of their own, with one, with some and with many; a sequence of no group
GROUPS = [(512, [515, 517, 600, 1500]), (0, [300])]


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def put_nan_keys(c, b, lo, hi, head):
    """Positions [lo, hi) of sequence b: keys of NaN in KV head `head`."""
    j = torch.arange(lo, hi, device=DEV)
    raw = c.pools[0].view(torch.uint8) if c.pools[0].dtype is torch.float8_e4m3fn else c.pools[0]
    raw[c.table[b, j // c.page].long(), head, j % c.page] = 0x7F if raw.dtype is torch.uint8 else float("nan")


def check(c, out, want, spoilt, status):
    """spoilt [batch, rows, h_q]: the rows that see a NaN score."""
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(torch.isnan(out), spoilt[..., None].expand(out.shape)), [
        (b, int(torch.isnan(out[b]).any(-1).sum()), int(spoilt[b].sum())) for b in range(out.shape[0])]
    for b, (w, tol) in enumerate(want):
        off = ((out[b].double() - w).abs() - tol)[~spoilt[b]]
        assert off.numel() == 0 or float(off.max()) <= 0, (b, float(off.max()))


def clean(c):
    return [c.expect(b) for b in range(len(c.lens_list))], torch.zeros(c.q.shape[:3], dtype=torch.bool, device=DEV)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,h_q,h_kv", VECTORS)
def test_a_nan_query(rows, h_q, h_kv, d, out, pool):
    """One element of one query vector, and whole vectors: with no own positions beside the prefix (rows == 1), and some."""
    groups = [(512, [511 + rows, 513, 600, 1500]), (0, [300])]
    c = Case(groups, rows, h_q, h_kv, d, 16, pool, out, d + rows)
    want, spoilt = clean(c)
    for b in range(len(c.lens_list)):
        r, h = b % rows, (3 * b) % h_q
        c.q[b, r, h, 5 if b % 2 else slice(None)] = float("nan")
        spoilt[b, r, h] = True
    if rows > 1:   # (a row that sees nothing sees no NaN; here every row sees a position)
        assert min(c.lens_list) >= rows
    status = ints([0])
    check(c, c.run(status=status), want, spoilt, status)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,h_q,h_kv", VECTORS)
@pytest.mark.parametrize("lo,hi", [(0, 128), (384, 512), (128, 256), (0, 512), (100, 101)])
def test_nan_keys_in_the_prefix(lo, hi, rows, h_q, h_kv, d, out, pool):
    """A split of the prefix, any of them, all of it, and one key: every row of the group's that belongs to the head."""
    c = Case(GROUPS, rows, h_q, h_kv, d, 16, pool, out, d + lo)
    want, spoilt = clean(c)
    put_nan_keys(c, 0, lo, hi, 1)
    spoilt[:4, :, h_q // h_kv:] = True
    status = ints([0])
    check(c, c.run(status=status), want, spoilt, status)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,h_q,h_kv", VECTORS)
def test_nan_keys_among_own_positions(rows, h_q, h_kv, d, out, pool):
    """Everything that a sequence does not share: its only own position, some hundred, a thousand (several splits), and all of
    a sequence of no group. Rows that see none of it stay as they are."""
    groups = [(512, [512 + rows - 1, 512 + rows, 650, 1500]), (0, [300])]
    c = Case(groups, rows, h_q, h_kv, d, 16, pool, out, d + 1)
    want, spoilt = clean(c)
    for b, n in enumerate(c.lens_list):
        lo = 512 if b < 4 else 0
        put_nan_keys(c, b, lo, n, 0)
        for r in range(rows):
            spoilt[b, r, : h_q // h_kv] = n - rows + r + 1 > lo
    assert not bool(spoilt[0, 0].any()) and bool(spoilt[1, 0].any())
    status = ints([0])
    check(c, c.run(status=status), want, spoilt, status)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,h_q", [(4, 8), (20, 4), (70, 6)])
def test_a_nan_key_and_a_nan_value_behind_earlier_rows(rows, h_q, d, out, pool):
    """The last row's own position holds a NaN key in one head and a NaN value in the other, and some rows before see only a
    NaN key among the own positions: a value that a row does not see spoils neither it nor the NaN that it does see."""
    c = Case([(512, [512 + rows - 1, 512 + rows + 40])], rows, h_q, 2, d, 16, pool, out, d + 2)
    want, spoilt = clean(c)
    half = h_q // 2
    for b, n in enumerate(c.lens_list):
        first = rows // 2                         # the first row that sees the NaN key, in head 0
        at = n - rows + first
        put_nan_keys(c, b, at, at + 1, 0)
        spoilt[b, first:, :half] = True
        v = c.pools[1].view(torch.uint8) if pool == "e4m3" else c.pools[1]
        v[c.table[b, (n - 1) // 16].long(), :, (n - 1) % 16] = 0x7F if pool == "e4m3" else float("nan")
        spoilt[b, rows - 1] = True                # in both heads
    status = ints([0])
    check(c, c.run(status=status), want, spoilt, status)
