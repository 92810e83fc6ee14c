"""Prompts with values that are not finite."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_prompt import check, expect, inputs, near, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


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
