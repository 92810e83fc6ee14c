"""Capped windows whose raw scores are large and their factor small: E4M3 pools with one scale, where a query enters
the product times 2^e, and bf16 keys far from one. Every score lies between 0.42 and 0.6 of the cap, as many of them
as make each nat of it weigh the same, so that an error in the cap's slope shows in the output.

Tolerance: relative 2-norm over a sequence. Values are random and independent of the weights, so weights off by e
change the output by e of its norm: 2^-8 a weight of an E4M3 window, 2^-17 a bf16 one. The queries are exact in their
terms (powers of two times a factor of a few bits); the score's own sum and the cap leave 2^-20 of a score of 30. A
bf16 output adds 2^-8.
"""

import math

import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.formats as of
import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


@pytest.mark.parametrize("cap", [50.0, 400.0])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("pool,block,log2", [("e4m3", 0, 0), ("bf16", 0, 15), ("bf16", 0, -9), ("e4m3", 64, 0)])
def test_scores_near_the_end_of_the_polynomial(pool, block, log2, d, cap):
    rows, h_q, h_kv, P, n = 16, 12, 2, 64, 1500
    g = np.random.default_rng(d)
    pages = -(-n // P)
    sign = g.choice([-1.0, 1.0], (h_kv, d))
    # keys of 448 and 320 by turns, the share of 448 set so that z falls from the top by an exponential of nats
    top, low = 0.59, 0.59 * 320 / 448
    fall = np.log1p(g.random(pages * P) * math.expm1(min(6.0, cap * (math.tanh(top) - math.tanh(low)))))
    x = np.arctanh(math.tanh(top) - fall / cap)
    share = np.clip((x / top * 448 - 320) / 128, 0.0, 1.0)
    mag = np.where(g.random((pages * P, h_kv, d)) < share[:, None, None], 448.0, 320.0) * sign
    keys = np.ascontiguousarray(mag.reshape(pages, P, h_kv, d).transpose(0, 2, 1, 3), dtype=np.float32)
    vals = g.standard_normal((pages, h_kv, P, d)).astype(np.float32)
    unit = 2.0 ** log2          # bf16 keys of 10^7, and near one
    codes = [of.encode(keys * np.float32(unit), pool), of.encode(vals, pool)]
    factor = g.choice([0.9375, 0.96875, 1.0], (rows, h_q))
    q = (2.0 * factor[..., None] * np.repeat(sign, h_q // h_kv, axis=0)).astype(np.float32)[None]
    scale = 1.0 / math.sqrt(d)
    k_scale = float(np.float32(top * cap / (scale * 2.0 * 448 * d * unit)))
    scales = [np.full((pages, h_kv, P // block), s, np.float32) for s in (k_scale, 1.0)] if block else [None, None]
    values = [oc.pool_values(c, pool, 1.0 if block else s, w) for c, s, w in zip(codes, (k_scale, 1.0), scales)]
    table, lens = np.arange(pages, dtype=np.int32)[None], np.array([n], dtype=np.int32)
    ref = oc.attention(q, *values, table, lens, scale, softcap=cap)
    on = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    dev = [on(c.view(np.int16)).view(torch.bfloat16) if pool == "bf16" else on(c) for c in codes]
    args = on(q).to(torch.bfloat16), *dev
    if block:
        call = lambda t: nbx.nbx_paged_decode_attn_block_scaled(*args, *map(on, scales), on(table), on(lens), n, scale,  # noqa: E731
                                                                softcap=cap, out_dtype=t)
    else:
        call = lambda t: nbx.nbx_paged_decode_attn_modified(*args, on(table), on(lens), n, scale, k_scale, 1.0,  # noqa: E731
                                                            softcap=cap, out_dtype=t)
    for t, bound in ((torch.bfloat16, 2.0 ** -8 + (2.0 ** -17 if pool == "bf16" else 2.0 ** -8)),
                     (torch.float32, 2.0 ** -17 if pool == "bf16" else 0.0)):
        got = call(t).double().cpu().numpy()
        off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert off <= bound + cap * 2.0 ** -19
