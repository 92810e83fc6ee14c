"""Decodes into an output that is aligned to 16 bytes and no more, as the calls ask for: the bits of any other output's, and
nothing beside it written."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def shifted(like, dtype):
    """(a whole buffer, an output of `like`'s shape 16 bytes into it)"""
    skip = 16 // dtype.itemsize
    whole = torch.full((like.numel() + 2 * skip,), 7.0, dtype=dtype, device=DEV)
    out = whole[skip:-skip].view(like.shape)
    assert out.data_ptr() % 32 == 16
    return whole, out, skip


# single-row decodes, windows of the tensor cores and, with 160 sequences, units of which each is a whole sequence
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[1, 100, 200, 256], [1000, 300, 513], [160] * 160], ids=["short", "mixed", "many"])
@pytest.mark.parametrize("rows,h_q,h_kv,d", [(1, 8, 2, 128), (16, 24, 4, 256), (8, 32, 4, 128), (128, 2, 1, 128), (70, 2, 1, 64)])
@pytest.mark.parametrize("call", ["plain", "modified", "bf16 output"])
def test_16_bytes(call, rows, h_q, h_kv, d, lens, pool):
    c = Case([(0, lens)], rows, h_q, h_kv, d, 64, pool, "f32", d + rows)
    k = dict(k_scale=c.scales[0], v_scale=c.scales[1])
    dtype = torch.bfloat16 if call == "bf16 output" else torch.float32
    decode = nbx.nbx_paged_decode_attn if call == "plain" else nbx.nbx_paged_decode_attn_modified
    args = (c.q, *c.pools, c.table, c.lens, c.max_len, c.scale)
    want = decode(*args, out=torch.empty(c.q.shape, dtype=dtype, device=DEV), **k)
    whole, out, skip = shifted(c.q, dtype)
    decode(*args, out=out, **k)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert bool((whole[:skip] == 7.0).all()) and bool((whole[-skip:] == 7.0).all())
    if call == "plain" and rows * h_q // h_kv >= 64 and d > 64:   # (the store that this is about)
        assert nbx.nbx_paged_decode_partial_kernel(nbx.NBX_BF16, nbx.dtype_code(c.pools[0]), rows, h_q, h_kv, d, c.num_pages,
                                                   64) != nbx.PARTIAL_SIMT
