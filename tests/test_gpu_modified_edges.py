"""Modified decodes at the ends of their sizes: more sequences than the plan keeps in shared memory on the tensor cores,
no position anywhere, no sequence, a long sequence of which a row sees a few keys. Tolerances:
tests/test_window_bounds.py, tests/test_gpu_modified.py."""

import numpy as np
import pytest
import torch

import oracle.cache as oc
import paged_split_kv_append_gb300 as nbx
from tests import test_gpu_modified as gm
from tests.test_window_bounds import bound, reference, relative

pytestmark = pytest.mark.gpu
DEV = gm.DEV


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    nbx.nbx_set_decode_grid_limit(0)


@pytest.mark.parametrize("pool,T", [("bf16", 0), ("e4m3", 0), ("block", 64)])
def test_windows_of_more_sequences_than_the_plan_sorts(pool, T):
    lens = np.random.default_rng(70).integers(0, 150, 2060)
    c = gm.Case(pool, "bf16", 10, 4, 1, 128, 64, lens, T, seed=70)
    assert gm.on_tensor_cores(c, "bf16")
    for mod in (dict(), dict(mask="random", softcap=4.0)):
        m = gm.made(mod, c.lens, 10, 4)
        ref = reference(c, **m)
        got = c.call("bf16", **m).double().cpu().numpy()
        off = relative(got, ref)
        assert max(off.values()) <= bound(c, "bf16")
        empty = np.all(ref == 0, axis=-1)
        assert np.all(got[empty] == 0)


@pytest.mark.parametrize("pool,T,rows", [("f32", 0, 1), ("bf16", 0, 1), ("block", 16, 1), ("bf16", 0, 32), ("block", 16, 32)])
def test_no_position_and_no_sequence(pool, T, rows):
    c = gm.Case(pool, "bf16", rows, 4, 1, 128, 64, (5, 9), T, seed=71)
    c.lens = np.zeros(2, dtype=np.int32)
    for out_type in ("f32", "bf16"):
        for mod in (dict(), dict(softcap=3.0, key_begin=np.zeros((2, rows)))):
            out = c.call(out_type, out=torch.full((2, rows, 4, 128), 7.0, dtype=gm.OUT[out_type], device=DEV), **mod)
            assert bool((out == 0).all())
    none = torch.zeros((0, rows, 4, 128), dtype=torch.bfloat16, device=DEV)
    table, lens = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((0, 3), 0))
    if pool == "block":
        s = [torch.from_numpy(x).to(DEV) for x in c.scales]
        out = nbx.nbx_paged_decode_attn_block_scaled(none, *c.dev, *s, table, lens, 64, 1.0)
    else:
        out = nbx.nbx_paged_decode_attn_modified(none, *c.dev, table, lens, 64, 1.0, softcap=2.0)
    assert out.shape == (0, rows, 4, 128)


@pytest.mark.parametrize("pool,T,rows", [("bf16", 0, 1), ("block", 16, 1), ("bf16", 0, 16), ("e4m3", 0, 16), ("f32", 0, 1)])
def test_a_few_keys_of_a_long_sequence(pool, T, rows):
    # one sequence of 131072 positions with one KV head; rows see 1 to 70 keys near its start, its middle, its end
    n = 131072
    c = gm.Case(pool, "f32" if pool == "f32" else "bf16", rows, 8, 1, 128, 64, (n,), T, seed=72)
    q = c.q.float().numpy()
    g = np.random.default_rng(73)
    for first in (0, 60000, n - 100):
        lo = first + g.integers(0, 30, (1, rows))
        hi = lo + g.integers(1, 70, (1, rows))
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = c.call("bf16", key_begin=lo, key_end=hi, status=status).double().cpu().numpy()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        ref = oc.attention(q, *c.values, c.table, c.lens, c.scale, key_begin=lo, key_end=hi)
        if rows == 1:
            assert np.abs(got - ref).max() <= c.tolerance("bf16")
        else:
            assert max(relative(got, ref).values()) <= bound(c, "bf16")
