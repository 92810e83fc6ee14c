"""The rotated append against its definition in 64 bits.

Tolerances. A turned element is r = a c - b s: one rounded product (2^-24 |a c|), one FMA (2^-24 |r|), then the product
with the reciprocal scale (2^-24 for it, 2^-24 for the reciprocal), then the cast: half a step of the output's type,
2^-24 (fp32: none further), 2^-8 (bf16: 7 bits behind the leading one, so a step is 2^-7 of the value's power of two and
half of it up to 2^-8 of the value) or 2^-4 relative for E4M3 (3 bits), 2^-10 absolute below 2^-6.
The cast of a value that is off by its fp32 error is off by at most both together.
"""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.uint8: 2.0 ** -4}


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def turn(x, cos, sin, positions, interleaved):
    """(turned x, the sum of the magnitudes of its terms) in 64 bits; x [n, h, d]."""
    x = x.double().cpu()
    half = cos.shape[1]
    c = cos.cpu().double()[positions.long().cpu()][:, None]
    s = sin.cpu().double()[positions.long().cpu()][:, None]
    y, mag = x.clone(), x.abs()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
        mag[..., a] = (x[..., a] * c[..., i]).abs() + y[..., a].abs()
        mag[..., b] = (x[..., b] * c[..., i]).abs() + y[..., b].abs()
    return y, mag


def values(t):
    return (t.view(torch.float8_e4m3fn) if t.dtype is torch.uint8 else t).double().cpu()


def near(got, want, mag, fp32_roundings):
    """Within the roundings of `want`'s fp32 evaluation and of the cast to got's type."""
    e4m3 = got.dtype is torch.uint8
    want, g = want.clamp(-448, 448) if e4m3 else want, values(got)
    room = fp32_roundings * 2.0 ** -24 * mag + HALF[got.dtype] * want.abs() * (1 + 2.0 ** -6) + (2.0 ** -10 if e4m3 else 0)
    assert torch.equal(torch.isnan(g), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert bool(((g - want).abs() <= room)[keep].all()), float(((g - want).abs() - room)[keep].max())


def case(n, h_q, h_kv, d, turned, page, new, pool, seed, fused=True, far=500):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, h_q + 2 * h_kv, d), generator=g, device=DEV).to(TYPES[new])
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    num_pages = max(1, -(-n // page)) + 2
    slots = torch.randperm(num_pages * page, generator=g, device=DEV)[:n].to(torch.int32)
    angle = torch.randn((far, turned // 2), generator=g, device=DEV, dtype=torch.float64) * 10
    positions = torch.randint(0, far, (n,), generator=g, device=DEV, dtype=torch.int32)
    fill = 0x7F if pool == "e4m3" else 7.0
    pools = [torch.full((num_pages, h_kv, page, d), fill, device=DEV).to(TYPES[pool]) for _ in range(2)]
    return q, k, v, angle.cos().float(), angle.sin().float(), positions, pools, slots


def check(q, k, v, cos, sin, positions, pools, before, slots, q_out, k_scale, v_scale, interleaved):
    torch.cuda.synchronize()
    page = pools[0].shape[2]
    if q is not None:
        near(q_out, *turn(q, cos, sin, positions, interleaved), 1)
    at = slots.long()
    kt, mag = turn(k, cos, sin, positions, interleaved)
    near(pools[0][at // page, :, at % page], kt / k_scale, mag / k_scale, 3)
    vt = v.double().cpu() / v_scale
    near(pools[1][at // page, :, at % page], vt, vt.abs(), 3)
    for p, b in zip(pools, before):       # nothing else is touched
        rest = torch.ones(p.shape[0] * page, dtype=torch.bool, device=DEV)
        rest[at] = False
        rows = torch.nonzero(rest)[:, 0]
        raw = torch.uint8 if p.dtype is torch.uint8 else torch.int16 if p.dtype is torch.bfloat16 else torch.int32
        assert torch.equal(p.view(raw)[rows // page, :, rows % page], b.view(raw)[rows // page, :, rows % page])


@pytest.mark.parametrize("new", ["f32", "bf16"])
@pytest.mark.parametrize("pool", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("d,turned", [(64, 64), (128, 32), (256, 256), (16, 16), (80, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_widths(new, pool, d, turned, interleaved):
    q, k, v, cos, sin, at, pools, slots = case(37, 6, 2, d, turned, 16, new, pool, d + turned)
    ks, vs = (0.02, 0.03) if pool == "e4m3" else (1.0, 1.0)
    before = [p.clone() for p in pools]
    status = ints([0])
    out = nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots, ks, vs, interleaved, status=status)
    check(q, k, v, cos, sin, at, pools, before, slots, out, ks, vs, interleaved)
    assert int(status) == 0


@pytest.mark.parametrize("n,h_q,h_kv", [(1, 1, 1), (1, 32, 8), (3, 5, 5), (31, 24, 4), (1000, 32, 8), (5003, 8, 1)])
@pytest.mark.parametrize("fused", [False, True])
def test_counts_and_strides(n, h_q, h_kv, fused):
    q, k, v, cos, sin, at, pools, slots = case(n, h_q, h_kv, 128, 128, 48, "bf16", "bf16", n, fused)
    before = [p.clone() for p in pools]
    out = nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots)
    check(q, k, v, cos, sin, at, pools, before, slots, out, 1.0, 1.0, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_in_place_and_keys_alone(interleaved):
    q, k, v, cos, sin, at, pools, slots = case(70, 4, 2, 64, 32, 16, "bf16", "bf16", 5)
    was, before = q.clone(), [p.clone() for p in pools]
    out = nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots, interleaved=interleaved, q_out=q)
    assert out is q
    check(was, k, v, cos, sin, at, pools, before, slots, q, 1.0, 1.0, interleaved)
    pools2 = [b.clone() for b in before]
    assert nbx.nbx_paged_kv_append_rotated(None, k, v, cos, sin, at, *pools2, slots, interleaved=interleaved) is None
    check(None, k, v, cos, sin, at, pools2, before, slots, None, 1.0, 1.0, interleaved)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, pools2))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
def test_turned_keys_beside_the_pool(interleaved, in_place, with_q):
    q, k, v, cos, sin, at, pools, slots = case(70, 4, 2, 64, 32, 16, "bf16", "e4m3", 15)
    slots[3] = -1                            # no place in the pool: its keys and queries are turned all the same
    was, before = k.clone(), [p.clone() for p in pools]
    k_out = k if in_place else torch.full_like(was, 9.0)
    out = nbx.nbx_paged_kv_append_rotated(q if with_q else None, k, v, cos, sin, at, *pools, slots, 0.02, 0.02, interleaved,
                                          k_out=k_out)
    near(k_out, *turn(was, cos, sin, at, interleaved), 1)
    if with_q:
        near(out, *turn(q, cos, sin, at, interleaved), 1)
    keep = torch.arange(70, device=DEV) != 3
    check(None, was[keep], v[keep], cos, sin, at[keep], pools, before, slots[keep], None, 0.02, 0.02, interleaved)


def test_an_angle_of_zero_is_the_plain_append():
    q, k, v, cos, sin, at, pools, slots = case(50, 4, 2, 128, 128, 16, "f32", "e4m3", 6, fused=False)
    plain = [p.clone() for p in pools]
    nbx.nbx_paged_kv_append_rotated(q, k, v, torch.ones_like(cos), torch.zeros_like(sin), at, *pools, slots, 0.02, 0.05)
    nbx.nbx_paged_kv_append(k, v, *plain, slots, 0.02, 0.05)
    assert torch.equal(pools[0], plain[0]) and torch.equal(pools[1], plain[1])


def test_saturation_and_values_that_are_not_finite():
    q, k, v, cos, sin, at, pools, slots = case(8, 2, 1, 64, 32, 16, "f32", "e4m3", 7)
    k[0, 0, 40], k[1, 0, 41], v[2, 0, 3], v[3, 0, 4], v[4, 0, 5] = 1e30, float("nan"), float("inf"), -1e9, float("nan")
    k[5, 0, 2] = float("nan")            # reaches its pair, and nothing else
    nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots)
    kt, _ = turn(k, cos, sin, at, False)
    s = slots.long()
    got = values(pools[0])[s.cpu() // 16, :, s.cpu() % 16]
    assert torch.equal(torch.isnan(got), torch.isnan(kt)) and int(torch.isnan(got).sum()) == 3
    assert float(got[0, 0, 40]) == 448.0
    got = values(pools[1])[s.cpu() // 16, :, s.cpu() % 16]
    assert float(got[2, 0, 3]) == 448.0 and float(got[3, 0, 4]) == -448.0 and bool(torch.isnan(got[4, 0, 5]))


def test_bad_slots_and_positions():
    q, k, v, cos, sin, at, pools, slots = case(9, 3, 2, 64, 64, 16, "bf16", "bf16", 8)
    total = pools[0].shape[0] * 16
    at[2], at[3] = -1, 500
    slots[4], slots[5] = -1, total
    before, status = [p.clone() for p in pools], ints([0])
    mark = torch.full((9, 3, 64), 9.0, device=DEV).to(torch.bfloat16)
    out = nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots, q_out=mark, status=status)
    assert int(status) == nbx.DEV_BAD_SLOT | nbx.DEV_BAD_LEN
    assert bool((out[2:4] == 9.0).all())
    fine = torch.tensor([0, 1, 4, 5, 6, 7, 8], device=DEV)
    near(out[fine], *turn(q[fine], cos, sin, at[fine], False), 1)
    fine = torch.tensor([0, 1, 6, 7, 8], device=DEV)
    check(None, k[fine], v[fine], cos, sin, at[fine], pools, before, slots[fine], None, 1.0, 1.0, False)


def test_far_offsets():
    """Token strides whose offsets pass 2^31 elements, and a pool behind them."""
    n, stride = 3, (1 << 30) + 64
    base = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device=DEV)
    k = torch.as_strided(base, (n, 1, 64), (stride, 64, 1))
    k.copy_(torch.randn((n, 1, 64), device=DEV))
    pools = [torch.zeros((1 << 21, 8, 128, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]   # 2^35 codes
    k16 = k[:, :, :16]
    k16 = torch.as_strided(base, (n, 1, 16), (stride, 16, 1)).expand(n, 8, 16).contiguous()
    cos, sin = torch.ones((4, 8), device=DEV), torch.zeros((4, 8), device=DEV)
    last = (1 << 21) * 128 - 1
    slots, at = ints([last, 5, last - 128 * 7]), ints([0, 1, 2])
    nbx.nbx_paged_kv_append_rotated(None, k16, k16, cos, sin, at, *pools, slots)
    s = slots.long()
    near(pools[0][s // 128, :, s % 128], k16.double().cpu(), k16.double().cpu().abs(), 3)
    near(pools[1][s // 128, :, s % 128], k16.double().cpu(), k16.double().cpu().abs(), 3)
    del pools
    pools = [torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    before = [p.clone() for p in pools]
    cos, sin = cos.repeat(1, 4), sin.repeat(1, 4)
    out = nbx.nbx_paged_kv_append_rotated(k, k, k, cos, sin, at, *pools, ints([3, 9, 20]))
    check(k, k, k, cos, sin, at, pools, before, ints([3, 9, 20]), out, 1.0, 1.0, False)


def test_another_stream_and_a_replayed_graph():
    q, k, v, cos, sin, at, pools, slots = case(64, 4, 2, 128, 128, 16, "bf16", "bf16", 10)
    before = [p.clone() for p in pools]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots, stream=side)
    torch.cuda.synchronize()
    check(q, k, v, cos, sin, at, pools, before, slots, out, 1.0, 1.0, False)
    out = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nbx.nbx_paged_kv_append_rotated(q, k, v, cos, sin, at, *pools, slots, q_out=out)
    q.mul_(-0.5)
    k.mul_(2)
    at.copy_((at + 1) % 500)
    graph.replay()
    torch.cuda.synchronize()
    check(q, k, v, cos, sin, at, pools, before, slots, out, 1.0, 1.0, False)


def test_refusals_of_the_binding():
    q, k, v, cos, sin, at, pools, slots = case(4, 2, 1, 64, 64, 16, "bf16", "bf16", 11)
    call = nbx.nbx_paged_kv_append_rotated
    for bad in (lambda: call(q.float(), k, v, cos, sin, at, *pools, slots), lambda: call(q, k.float(), v, cos, sin, at, *pools, slots),
                lambda: call(q, k, v, cos, sin, at[:3], *pools, slots), lambda: call(q, k, v, cos, sin, at, *pools, slots[:3]),
                lambda: call(q, k, v, cos.double(), sin, at, *pools, slots), lambda: call(q, k, v, cos, sin[:-1], at, *pools, slots),
                lambda: call(q, k, v, cos, sin, at.long(), *pools, slots), lambda: call(q[:3], k, v, cos, sin, at, *pools, slots),
                lambda: call(q.transpose(0, 1), k, v, cos, sin, at, *pools, slots), lambda: call(q, k[..., :32], v[..., :32], cos, sin, at, *pools, slots),
                lambda: call(None, k, v, cos, sin, at, *pools, slots, q_out=q),
                lambda: call(q, k, v, cos, sin, at, *pools, slots, k_out=q),
                lambda: call(q, k, v, cos, sin, at, *pools, slots, k_out=k.float()),
                lambda: call(q, k, v, cos, sin, at, *pools, slots, status=at[4:]),
                lambda: call(q, k, v, cos, sin, at, pools[0], pools[1][:1], slots),
                lambda: call(q, k, v, cos.cpu(), sin, at, *pools, slots)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nbx.NbxError):       # 24 elements turned
        call(q, k, v, cos[:, :12].contiguous(), sin[:, :12].contiguous(), at, *pools, slots)
    wide = torch.zeros((4, 4 * 64 + 4), dtype=torch.bfloat16, device=DEV)   # rows that start off 16 bytes
    with pytest.raises(nbx.NbxError):
        call(None, wide[:, :64].view(4, 1, 64), wide[:, 64:128].view(4, 1, 64), cos, sin, at, *pools, slots)
    empty = call(q[:0], k[:0], v[:0], cos, sin, at[:0], *pools, slots[:0])
    assert empty.shape == (0, 2, 64)
