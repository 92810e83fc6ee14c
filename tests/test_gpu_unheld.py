"""What a page holds at positions that no sequence holds is nobody's: outputs have the same bits whether it is zero,
large, or not a number."""

import numpy as np
import pytest
import torch

import oracle.cache as oc
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


@pytest.mark.parametrize("out_type", ["f32", "bf16"])
@pytest.mark.parametrize("pool,rows,h_q,h_kv,d,P,T", SHAPES)
def test_keys_behind_a_sequence_under_a_cap(pool, rows, h_q, h_kv, d, P, T, out_type):
    # scores within the cap's polynomial: a key that nobody sees may not choose the form that they take
    c = Case(pool, "bf16", rows, h_q, h_kv, d, P, LENS, T, seed=41)
    for cap in (12.0, 100.0):
        out = []
        for what in ("zero", "large", "nan"):
            c.dev = filled(c, what)
            out.append(c.call(out_type, softcap=cap))
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("pool,T", [("bf16", 0), ("e4m3", 0), ("block", 16)])
def test_a_cap_does_not_see_the_other_rows(pool, T):
    # rows of small scores beside one of large ones, a large cap: what it leaves of a small score is the score, to
    # 2^-21 of the score itself and not of the cap. Tolerance as in test_gpu_unmodified (fp32 sums), weights 2^-17
    rows, h_q, h_kv, d, P = 16, 16, 2, 128, 64
    c = Case(pool, "bf16", rows, h_q, h_kv, d, P, (700,), T, seed=42)
    q = c.q.float()
    q[0, ::5] *= 3e6
    c.q = q.to(torch.bfloat16)
    cap = 1e5
    ref = oc.attention(c.q.float().numpy(), *c.values, c.table, c.lens, c.scale, softcap=cap)
    quiet = [r for r in range(rows) if r % 5]
    z = c.scale * float(np.linalg.norm(c.q.float().numpy()[0, quiet], axis=-1).max()) * \
        float(np.linalg.norm(c.values[0], axis=-1).max())
    got = c.call("f32", softcap=cap).double().cpu().numpy()
    off = np.linalg.norm(got[0, quiet] - ref[0, quiet]) / np.linalg.norm(ref[0, quiet])
    assert off <= 2.0 ** -17 + 2.0 ** -19 * z + 2.0 ** -14, off
