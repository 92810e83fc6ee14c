"""Modified windows sequence by sequence: the relative 2-norm of a sequence's outputs, which a batch's largest value
does not widen. A merge that loses a split, or a kernel that writes zeros, is far outside: planted in the definition,
on the host, below.

Tolerance. Values are random and independent of the weights, so relative errors of the weights of at most e change a
sequence's outputs by at most e of their norm (for a single key by e itself). On tensor cores an E4M3 pool's weights are
held to 2^-8, a bf16 pool's to 2^-17, and each element of an E4M3 window's queries to 2^-16 of the vector's largest: the
d roundings of a score, independent of one another, move it by 2^-16 scale max|q| |k|. The score's own sum is off by
2^-20 Z, Z = scale |q| |k|, sums of weights and values by 2^-15 at most, and a bf16 output by 2^-8."""

import numpy as np
import pytest
import torch

import oracle.cache as oc
import paged_split_kv_append_gb300 as nbx
from tests import test_gpu_modified as gm

WEIGHT = {"bf16": 2.0 ** -17, "e4m3": 2.0 ** -8, "block": 2.0 ** -8}


def relative(got, ref):
    """The relative 2-norm of every sequence that has outputs, by its number."""
    return {b: float(np.linalg.norm(got[b] - ref[b]) / np.linalg.norm(ref[b])) for b in range(len(ref)) if ref[b].any()}


def bound(c, out_type):
    q, k = c.q.float().numpy(), float(np.linalg.norm(c.values[0], axis=-1).max())
    z = c.scale * float(np.linalg.norm(q, axis=-1).max()) * k
    query = 0.0 if c.pool == "bf16" else 2.0 ** -16 * c.scale * float(np.abs(q).max()) * k
    return WEIGHT[c.pool] + query + 2.0 ** -19 * z + 2.0 ** -14 + (2.0 ** -8 if out_type == "bf16" else 0.0)


def reference(c, **mod):
    return oc.attention(c.q.float().numpy(), *c.values, c.table, c.lens, c.scale, **mod)


@pytest.mark.gpu
@pytest.mark.parametrize("mod", gm.MODS, ids=lambda m: "-".join(str(v) for v in m.values()) or "plain")
@pytest.mark.parametrize("pool,rows,h_q,h_kv,d,P,T", gm.TENSOR)
def test_every_sequence_of_a_window(pool, rows, h_q, h_kv, d, P, T, mod):
    nbx.build()
    c = gm.Case(pool, "bf16", rows, h_q, h_kv, d, P, gm.WINDOW_LENS + (3000,), T, seed=60, two=(rows != 8))
    m = gm.made(mod, c.lens, rows, h_q)
    ref = reference(c, **m)
    for out_type in ("bf16", "f32") if pool == "bf16" else ("bf16",):
        assert gm.on_tensor_cores(c, out_type)
        off = relative(c.call(out_type, **m).double().cpu().numpy(), ref)
        worst = max(off, key=off.get)
        assert off[worst] <= bound(c, out_type), f"{c.lens[worst]} positions: {off[worst]:.3g} of {bound(c, out_type):.3g}"


@pytest.mark.parametrize("cap", [0.0, 2.0])
@pytest.mark.parametrize("pool,rows,h_q,h_kv,d,P,T", [s for s in gm.TENSOR if s[1] <= 16])
def test_the_bound_sees_a_lost_split_and_zeros(monkeypatch, pool, rows, h_q, h_kv, d, P, T, cap):
    monkeypatch.setattr(gm, "DEV", "cpu")
    c = gm.Case(pool, "bf16", rows, h_q, h_kv, d, P, (513, 1100, 3000), T, seed=60, two=(rows != 8))
    ref = reference(c, softcap=cap)
    assert all(off > 10 * bound(c, "bf16") for off in relative(np.zeros_like(ref), ref).values())
    # without its first 256 positions: a split of the last sequence's, or the shortest there is
    late = np.full((3, rows), 256)
    lost = relative(reference(c, softcap=cap, key_begin=late), ref)
    assert len(lost) == 3 and all(off > 4 * bound(c, "bf16") for off in lost.values()), (lost, bound(c, "bf16"))
