"""What the bindings of the cache operators refuse beside shapes and types: a status word without an element (the call's
findings would be lost), and a block-scaled call without scales."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


def test_a_status_word_without_an_element():
    none = i32(4)[4:]
    pool = [torch.zeros((4, 1, 16, 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones((4, 1, 1), device=DEV) for _ in range(2)]
    x, q = torch.zeros((1, 1, 64), device=DEV), torch.zeros((1, 1, 1, 64), device=DEV)
    table, one = i32(1, 4), i32(1)
    calls = [lambda s: nbx.nbx_paged_kv_append_block_scaled(x, x, *pool, *scales, table, one, i32(2), status=s),
             lambda s: nbx.nbx_paged_decode_attn_block_scaled(q, *pool, *scales, table, one, 16, 1.0, status=s),
             lambda s: nbx.nbx_paged_decode_attn_modified(q, *pool, table, one, 16, 1.0, softcap=1.0, status=s),
             lambda s: nbx.nbx_paged_kv_copy_pages(i32(1, 3), one, *pool, *scales, status=s),
             lambda s: nbx.nbx_paged_kv_fork(table, one, one, one, *pool, *scales, status=s),
             lambda s: nbx.nbx_paged_kv_compact(table, one, *pool, *scales, status=s)]
    for call in calls:
        with pytest.raises(ValueError, match="status"):
            call(none)
        call(i32(1))
    torch.cuda.synchronize()


def test_block_scaled_calls_without_scales():
    pool = [torch.zeros((4, 1, 16, 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    x, q = torch.zeros((1, 1, 64), device=DEV), torch.zeros((1, 1, 1, 64), device=DEV)
    with pytest.raises(ValueError, match="scales"):
        nbx.nbx_paged_kv_append_block_scaled(x, x, *pool, None, None, i32(1, 4), i32(1), i32(2))
    with pytest.raises(ValueError, match="scales"):
        nbx.nbx_paged_decode_attn_block_scaled(q, *pool, None, None, i32(1, 4), i32(1), 16, 1.0)
