"""A shared prefix of more than 2^30 positions, over a few pages that its row names again and again."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_shared import ints

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


@pytest.mark.parametrize("h_q", [1, 8])   # own positions by the one-warp kernel, and in the tiles
def test_positions_past_2_to_the_30(h_q):
    """Scores of 0 and values of -1 up to 2^30, of 32 and 1 behind: 2^30 weights of 1 beside 196608 of e^32 = 2^46, so the
    result is 1 to 2^-32 of it. Own positions have scores of 0."""
    page, far = 1 << 16, 3
    n = (1 << 30) + far * page
    pools = [torch.zeros((4, 1, page, 64), device=DEV) for _ in range(2)]
    pools[0][1, :, :, 0] = 32.0
    pools[1].fill_(-1.0)
    pools[1][1] = 1.0
    pools = [x.to(torch.float8_e4m3fn) for x in pools]
    table = torch.zeros((2, n // page + 1), dtype=torch.int32, device=DEV)
    table[:, (1 << 30) // page:] = 1
    table[:, -1] = ints([2, 3])
    q = torch.zeros((2, 1, h_q, 64), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    status = ints([0])
    out = nbx.nbx_paged_decode_attn_shared(q, *pools, table, ints([n + 17, n + 30]), n + 30, ints([0, 2]), ints([n]), 1.0,
                                           status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    # the sum of 2^30 and more weights, each term within 2^-24 of its place: far within this
    assert float((out - 1.0).abs().max()) < 2.0 ** -8


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_as_many_equal_weights(pool):
    """2^30 weights of 1 and values of -1. Of a split, 2^25 and more positions, sums of whole tiles are exact in fp32 up to
    2^31; joined and divided, they are off by a few 2^-24."""
    page = 1 << 16
    n = 1 << 30
    pools = [torch.zeros((3, 1, page, 64), device=DEV) for _ in range(2)]
    pools[1].fill_(-1.0)
    pools = [x.to(torch.float8_e4m3fn if pool == "e4m3" else torch.bfloat16) for x in pools]
    table = torch.zeros((2, n // page + 1), dtype=torch.int32, device=DEV)
    table[:, -1] = ints([1, 2])
    q = torch.zeros((2, 1, 1, 64), dtype=torch.bfloat16, device=DEV)
    out = nbx.nbx_paged_decode_attn_shared(q, *pools, table, ints([n + 17, n + 30]), n + 30, ints([0, 2]), ints([n]), 1.0)
    assert float((out + 1.0).abs().max()) < 2.0 ** -20
