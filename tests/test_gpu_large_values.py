"""Values near the type's largest: what a row adds up stays in fp32's range wherever weights of at most 1 leave it there.
Tolerances are those of test_gpu_prompt.py and test_gpu_shared.py, relative to the values."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_prompt import check, inputs, starts
from test_gpu_shared import Case, ints

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# The first tile of keys has scores of 0, the others this: less than the step of 2^8 at which a running maximum moves. 384
# values of 2^118 with weights of at most 1 sum to less than 2^127, with weights of e^5.1875 = 2^7.48 to over 2^132.
LATER, LARGE = 5.1875, 2.0 ** 118


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def large(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (LARGE * (0.5 + 0.5 * torch.rand(shape, generator=g, device=DEV))).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts(d):
    lens = [384, 130, 1]
    q, k, v = inputs(sum(lens), 4, 2, d, d, fused=False)
    q.zero_()
    q[:, :, 0] = 1.0
    k.zero_()
    for lo in (0, 384):
        k[lo + 128:lo + 384, :, 0] = LATER
    v.copy_(large(v.shape, d))
    check(q, k, v, lens, 1.0, nbx.nbx_prompt_attn(q, k, v, starts(lens), 1.0))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,h_q", [(1, 8), (2, 32)])
def test_shared(rows, h_q, d, out):
    """Enough of them that a split holds several tiles of keys, prefixes (2 query vectors to a KV head) and own positions."""
    groups = [(368, [370, 384]) for _ in range(40)] + [(0, [384]) for _ in range(20)]
    c = Case(groups, rows, h_q, 8, d, 16, "bf16", out, d)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.scale = 1.0
    k, v = c.pools
    k.zero_()
    v.copy_(large(v.shape, d + 1))
    t = c.table.long()[:, 8:]   # pages from position 128 on
    k[t[t >= 0].unique(), :, :, 0] = LATER
    c.poison()
    status = ints([0])
    c.check(c.run(status=status))
    assert int(status) == 0
