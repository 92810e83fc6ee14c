"""Values that are not finite, in prompts and among own positions. Rows that see them are done as quickly as any other; rows
that merely share a key tile with them are computed again, however long that takes."""

import math

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_prompt import check, expect, inputs, ints, near, starts
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")
LIMIT_NS = 20_000_000   # the calls below take about 1 ms


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    yield
    nbx.nbx_set_decode_wait_test(0, 0)


def call_with_limit(q, k, v, n, scale):
    """A call whose waits may take 20 ms. (Every wait is bounded: one that ran out would set a bit, and the call return.)"""
    status = ints([0])
    nbx.nbx_set_decode_wait_test(LIMIT_NS, 0)
    out = nbx.nbx_prompt_attn(q, k, v, starts([n]), scale, status=status)
    torch.cuda.synchronize()
    nbx.nbx_set_decode_wait_test(0, 0)
    assert int(status) == 0
    return out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_a_value_that_every_row_sees(d, bad):
    """16384 rows that all see the value of the first key: not one is computed again."""
    n, scale = 16384, 1 / math.sqrt(d)
    q, k, v = inputs(n, 8, 1, d, d, fused=False)
    v[0, 0, 7] = bad
    out = call_with_limit(q, k, v, n, scale)
    assert bool((torch.isnan(out[:, :, 7]) if bad != bad else out[:, :, 7] == bad).all())
    rows = [0, 1, 127, 128, 5000, n - 1]
    near(out[rows], *expect(q, k, v, 0, n, scale, rows))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_value_behind_the_rows_of_its_tile(d):
    """The last key's value: the rows before it in the last tile of keys, which do not see it, are computed again over all
    their 16384 keys, while the units behind them wait."""
    n, scale = 16384, 1 / math.sqrt(d)
    q, k, v = inputs(n, 8, 1, d, d, fused=False)
    v[n - 1, 0, 7] = NAN
    out = call_with_limit(q, k, v, n, scale)
    assert bool(torch.isnan(out[n - 1, :, 7]).all())
    rows = [0, 5000, n - 129, n - 128, n - 100, n - 2, n - 1]
    near(out[rows], *expect(q, k, v, 0, n, scale, rows))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(2, 2), (8, 1), (6, 2)])
def test_several_in_a_tile(d, h_q, h_kv):
    """Of both signs in one column, of several columns, at the first and the last key of a tile, in one head of several; NaN
    and infinite keys beside them."""
    lens = [1, 200, 300, 129]
    q, k, v = inputs(sum(lens), h_q, h_kv, d, 31, fused=False)
    v[0, 0, 0] = INF
    for at, head, column, bad in ((1, 0, 3, INF), (60, 0, 3, -INF), (128, 0, 9, NAN), (129, h_kv - 1, d - 1, INF),
                                  (200, 0, 1, -INF), (201, 0, 0, NAN), (328, 0, 2, INF), (329, h_kv - 1, 4, INF), (629, 0, 5, NAN)):
        v[at, head, column] = bad
    k[250, h_kv - 1, 6] = NAN
    check(q, k, v, lens, 0.1, nbx.nbx_prompt_attn(q, k, v, starts(lens), 0.1))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_without_a_score_beside_such_values(d):
    """Every score of the first 150 rows is -inf: they are 0, whatever their values and those behind them are."""
    q, k, v = inputs(200, 2, 1, d, 13, fused=False)
    q.fill_(1.0)
    k[:150, 0, 0] = -INF
    v[20, 0, 3], v[140, 0, 4], v[199, 0, 5] = NAN, INF, -INF
    out = nbx.nbx_prompt_attn(q, k, v, starts([200]), 0.1)
    assert bool((out[:150] == 0).all())
    want, tol = expect(q, k, v, 0, 200, 0.1, list(range(150, 200)))
    near(out[150:], want, tol)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_own_positions_that_every_row_sees(pool, d):
    """Windows of 64 rows behind 3000 positions, two units an SM and more: the fourth position holds such a value, and none of
    the rows, of which the earlier ones do not see the last positions, is computed again."""
    c = Case([(0, [3000])] * 160, 64, 8, 2, d, 64, pool, "f32", d)
    v = c.pools[1].view(torch.uint8) if pool == "e4m3" else c.pools[1]
    first = c.table[:, 0].long()
    v[first, 0, 3, 7] = 0x7F if pool == "e4m3" else INF
    v[first[::2], 1, 3, 9] = 0x7F if pool == "e4m3" else -INF
    out, status = torch.empty_like(c.q, dtype=torch.float32), ints([0])
    ws = torch.empty(nbx.nbx_paged_decode_shared_workspace_bytes(160, 64, 8, 2, d, c.max_len, 160), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    nbx.nbx_set_decode_wait_test(2_000_000, 0)   # (the call takes less)
    c.run(out=out, workspace=ws, status=status)
    torch.cuda.synchronize()
    nbx.nbx_set_decode_wait_test(0, 0)
    assert int(status) == 0
    odd = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    odd[:, :, :4, 7] = True
    odd[::2, :, 4:, 9] = True
    assert torch.equal(torch.isfinite(out), ~odd)
    v[first, 0, 3, 7] = v[first[::2], 1, 3, 9] = 0
    for b in (0, 1, 158, 159):
        want, tol = c.expect(b)
        assert bool((((out[b].double() - want).abs() <= tol) | odd[b]).all())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_own_positions_behind_earlier_rows(pool, d):
    """Such a value at the last of 3000 positions: 63 of the 64 rows are computed again, while the units behind them wait."""
    c = Case([(0, [3000])] * 160, 64, 8, 2, d, 64, pool, "f32", d)
    v = c.pools[1].view(torch.uint8) if pool == "e4m3" else c.pools[1]
    at, off = c.table[:, 2999 // 64].long(), 2999 % 64
    v[at, :, off, 7] = 0x7F if pool == "e4m3" else NAN
    out, status = torch.empty_like(c.q, dtype=torch.float32), ints([0])
    ws = torch.empty(nbx.nbx_paged_decode_shared_workspace_bytes(160, 64, 8, 2, d, c.max_len, 160), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    nbx.nbx_set_decode_wait_test(2_000_000, 0)
    c.run(out=out, workspace=ws, status=status)
    torch.cuda.synchronize()
    nbx.nbx_set_decode_wait_test(0, 0)
    assert int(status) == 0
    odd = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    odd[:, 63, :, 7] = True
    assert torch.equal(torch.isfinite(out), ~odd)
    v[at, :, off, 7] = 0
    for b in (0, 1, 158, 159):
        want, tol = c.expect(b)
        assert bool((((out[b].double() - want).abs() <= tol) | odd[b]).all())
