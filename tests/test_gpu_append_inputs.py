"""Block-scaled appends whose inputs another program made: held scales that are no powers of two, and token ranges
that do not ascend."""

import numpy as np
import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from tests.test_gpu_block_append import DEV, Cache, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_held_scales_that_are_no_powers_of_two(dtype):
    # a scale that another program wrote (amax / 448), new values beside the grid's ties: x / S, not x * (1 / S)
    B, P, T, h, d = 300, 16, 16, 2, 64
    table, pages = table_for([16] * B, P, 60)
    c = Cache(pages, h, P, d, T, 61)
    g = np.random.default_rng(62)
    for w in range(2):
        c.scales[w] = g.uniform(0.5, 8.0, c.scales[w].shape).astype(np.float32)
        c.dev_scales[w] = torch.from_numpy(c.scales[w].copy()).to(DEV)
    x = []
    for w in range(2):
        tie = (2 * g.integers(8, 16, (B * 6, h, d)) + 1) / 16.0 * np.exp2(g.integers(-6, 7, (B * 6, h, d)))
        s = np.repeat(c.scales[w][table[:, 0], :, 0], 6, axis=0)[..., None]
        x.append(torch.from_numpy((tie * s * g.choice([-1.0, 1.0], tie.shape)).astype(np.float32)).to(dtype).to(DEV))
    c.append(x, table, [5] * B, list(range(0, 6 * B + 1, 6)))
    c.check()


@pytest.mark.parametrize("start,bits", [([0, 1000, 0, 10], nbx.DEV_BAD_LEN), ([1000, 5, 6, 7], nbx.DEV_BAD_LEN),
                                        ([0, 1000, 1005, 1010], 0), ([0, 1000, 1000, 1000], 0), ([3, 3, 4, 4], 0)])
def test_ranges_that_do_not_ascend_are_reported(start, bits):
    # [0, 1000, 0, 10]: the blocks of the first sequence from the fifth on belong to nobody
    P, T, h, d = 16, 16, 1, 64
    table, pages = table_for([1100, 20, 20], P, 63)
    c = Cache(pages, h, P, d, T, 64)
    x = [torch.randn((1010, h, d), device=DEV) for _ in range(2)]
    dt = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)   # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nbx.nbx_paged_kv_append_block_scaled(*x, *c.dev, *c.dev_scales, dt(table), dt([0, 0, 0]), dt(start), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == bits
