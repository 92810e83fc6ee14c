"""What a page holds at positions that no sequence holds is nobody's: outputs have the same bits whether it is zero,
large, or not a number."""

import numpy as np
import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from tests.test_gpu_modified import DEV, Case, made

pytestmark = pytest.mark.gpu
# windows on the tensor cores (40 and 42 vectors: tile rows without a vector), single rows and small windows of one warp
SHAPES = [("bf16", 10, 16, 4, 128, 64, 0), ("e4m3", 10, 16, 4, 128, 64, 0), ("block", 7, 12, 2, 256, 64, 16),
          ("bf16", 1, 8, 2, 128, 16, 0), ("e4m3", 3, 8, 2, 64, 32, 0), ("block", 1, 32, 8, 128, 64, 16),
          ("block", 2, 6, 1, 256, 16, 16)]
LENS = (1, 7, 33, 70, 130, 500, 1003)


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    nbx.nbx_set_decode_grid_limit(0)


def filled(c, what):
    """The pools with every position that no sequence holds filled."""
    held = np.zeros((c.num_pages, c.P), dtype=bool)
    for b, n in enumerate(c.lens):
        for j in range(int(n)):
            held[c.table[b, j // c.P], j % c.P] = True
    free = torch.from_numpy(~held).to(DEV)[:, None, :, None]
    value = {"zero": 0.0, "large": 3e4, "nan": float("nan")}[what]
    code = {"zero": 0, "large": 0x7E, "nan": 0x7F}[what]
    return [torch.where(free, torch.full_like(t, value if t.dtype == torch.bfloat16 else code), t) for t in c.dev]


@pytest.mark.parametrize("out_type", ["f32", "bf16"])
@pytest.mark.parametrize("mod", [dict(), dict(mask="window"), dict(slopes=True)],
                         ids=lambda m: "-".join(str(v) for v in m) or "plain")
@pytest.mark.parametrize("pool,rows,h_q,h_kv,d,P,T", SHAPES)
def test_values_behind_a_sequence(pool, rows, h_q, h_kv, d, P, T, mod, out_type):
    c = Case(pool, "bf16", rows, h_q, h_kv, d, P, LENS, T, seed=40)
    out = []
    for what in ("zero", "large", "nan"):
        c.dev = filled(c, what)
        out.append(c.call(out_type, **made(mod, LENS, rows, h_q)))
    assert bool(torch.isfinite(out[0]).all())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
