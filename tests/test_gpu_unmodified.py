"""nbx_paged_decode_attn_modified without a modification: on windows, the plain decode's bits from a bf16 pool, and
fp32 sums from an E4M3 pool under an fp32 output, whatever the length.

Tolerance for E4M3: relative 2-norm over a sequence. A score is a sum of d exact products rounded at most 16 times on
its way, so off by 2^-20 Z, Z = scale |q| |k|; sums of weights and values are fp32 (at most 512 terms and 64 splits,
2^-14.8 in the worst case)."""

import numpy as np
import pytest
import torch

import oracle.cache as oc
import paged_split_kv_append_gb300 as nbx
from tests.test_gpu_modified import DEV, Case

pytestmark = pytest.mark.gpu
SHAPES = [(16, 24, 4, 256, 64), (8, 32, 4, 128, 128), (70, 12, 4, 128, 64), (128, 2, 1, 128, 64)]
LENS = [(0, 1, 100, 200, 255, 256, 257), (1000, 300, 513), (2500,), (160,) * 30]


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    nbx.nbx_set_decode_grid_limit(0)


@pytest.mark.parametrize("lens", LENS, ids=["short", "mixed", "long", "many"])
@pytest.mark.parametrize("rows,h_q,h_kv,d,P", SHAPES)
def test_a_bf16_window_is_the_plain_decode(rows, h_q, h_kv, d, P, lens):
    c = Case("bf16", "bf16", rows, h_q, h_kv, d, P, lens, seed=31)
    i32 = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    plain = nbx.nbx_paged_decode_attn(c.q.to(DEV), *c.dev, i32(c.table), i32(c.lens), int(c.lens.max()), c.scale)
    assert torch.equal(plain, c.call())


@pytest.mark.parametrize("lens", LENS, ids=["short", "mixed", "long", "many"])
@pytest.mark.parametrize("rows,h_q,h_kv,d,P", SHAPES)
def test_an_e4m3_window_with_an_fp32_output_keeps_fp32_weights(rows, h_q, h_kv, d, P, lens):
    c = Case("e4m3", "bf16", rows, h_q, h_kv, d, P, lens, seed=32)
    assert nbx.nbx_paged_decode_modified_partial_kernel(nbx.NBX_BF16, nbx.NBX_E4M3, nbx.NBX_F32, rows, h_q, h_kv, d,
                                                        c.num_pages, P) == nbx.PARTIAL_WARP
    ref = oc.attention(c.q.float().numpy(), *c.values, c.table, c.lens, c.scale)
    z = c.scale * float(np.linalg.norm(c.q.float().numpy(), axis=-1).max()) * \
        float(np.linalg.norm(c.values[0], axis=-1).max())
    for mod in (dict(), dict(softcap=1e6)):
        got = c.call(**mod).double().cpu().numpy()
        for b, n in enumerate(c.lens):
            if n:
                off = np.linalg.norm(got[b] - ref[b]) / np.linalg.norm(ref[b])
                assert off <= 2.0 ** -19 * z + 2.0 ** -14, f"{n} positions: {off:.3g}"
