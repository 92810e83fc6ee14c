"""Prompt attention against its definition in 64 bits.

Tolerance of an output o = sum a_j v_j, with M = sum a_j |v_j| (a: the exact weights):
- the output's own rounding to bf16 is half a step, up to 2^-8 |o|;
- each weight may be rounded to bf16 before its product, 2^-8 a_j at most: 2^-8 M;
- a score's fp32 sum of d exact products is off by at most d 2^-23 S, S = scale sum |q_i k_i| (one 2^-23 for each of d
  additions, for an accumulation that truncates), its factor and the difference to the maximum by 2^-23 of the
  largest |z| each, and exp2 by 2^-21: a weight is off by E = d 2^-23 S + 2^-22 max |z| + 2^-21 of itself, numerator
  and denominator: 2 E M. Sums over the keys add 2^-23 each, n 2^-23 M at most.
"""

import math

import pytest
import torch

import paged_split_kv_append_gb300 as nbx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def starts(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return ints(at)


def inputs(n, h_q, h_kv, d, seed, fused=True, spread=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, h_q + 2 * h_kv, d), generator=g, device=DEV)
    x *= torch.exp(spread * torch.randn((n, h_q + 2 * h_kv, 1), generator=g, device=DEV))
    x = x.to(torch.bfloat16)
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def expect(q, k, v, lo, hi, scale, rows=None):
    """(outputs, tolerances) of rows `rows` (all by default) of the sequence [lo, hi), in 64 bits."""
    h_q, h_kv, d = q.shape[1], k.shape[1], q.shape[2]
    G = h_q // h_kv
    at = torch.arange(hi - lo, device=DEV) if rows is None else torch.as_tensor(rows, device=DEV)
    qq = q[lo:hi][at].double().view(-1, h_kv, G, d)
    kk, vv = k[lo:hi].double(), v[lo:hi].double()
    z = torch.einsum("rhgd,jhd->rhgj", qq, kk) * scale
    dark = (torch.arange(hi - lo, device=DEV) > at[:, None])[:, None, None]
    z = z.masked_fill(dark, -math.inf)
    a = torch.softmax(z, -1)
    a = torch.where(z.amax(-1, keepdim=True) == -math.inf, torch.zeros_like(a), a)
    vv = vv.permute(1, 0, 2)[None]                                   # [1, h, j, d]
    seen = torch.where(dark[..., None], torch.zeros((), dtype=torch.float64, device=DEV), vv[:, :, None]) \
        if not bool(torch.isfinite(vv).all()) else None
    o = torch.einsum("rhgj,rhgjd->rhgd", a, seen.expand(*a.shape, d)) if seen is not None else \
        torch.einsum("rhgj,hjd->rhgd", a, vv[0])
    M = torch.einsum("rhgj,hjd->rhgd", a.nan_to_num(0.0), vv[0].abs().nan_to_num(0.0, 0.0, 0.0))
    S = (torch.einsum("rhgd,jhd->rhgj", qq.abs(), kk.abs()) * abs(scale)).masked_fill(dark, 0.0).nan_to_num(0.0, 0.0, 0.0)
    big = z.masked_fill(dark, 0.0).abs().nan_to_num(0.0, 0.0, 0.0).amax(-1, keepdim=True)
    E = d * 2.0 ** -23 * S.amax(-1, keepdim=True) + 2.0 ** -22 * big + 2.0 ** -21
    tol = 2.0 ** -8 * (o.abs().nan_to_num(0.0, 0.0, 0.0) + M) * (1 + 2.0 ** -7) + (2 * E + (hi - lo) * 2.0 ** -23) * M
    return o.reshape(-1, h_q, d), tol.reshape(-1, h_q, d)


def near(got, want, tol):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (int(torch.isnan(got).sum()), int(torch.isnan(want).sum()))
    same = (got == want) | torch.isnan(want)                          # infinities
    off = ((got - want).abs() - tol).masked_fill(same, -1.0)
    assert float(off.max()) <= 0.0, (float(off.max()), int((off > 0).sum()), off.numel())


def check(q, k, v, lens, scale, out, first=0):
    torch.cuda.synchronize()
    lo = first
    for n in lens:
        if n:
            near(out[lo:lo + n], *expect(q, k, v, lo, lo + n, scale))
        lo += n


LENS = [[1], [2, 1, 3], [17], [127, 128, 129], [0, 5, 0, 0, 64, 0], [255, 256, 257], [31, 32, 33, 63, 65], [300, 1, 511],
        [640]]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(d, lens):
    q, k, v = inputs(sum(lens), 8, 2, d, sum(lens) + d)
    out = nbx.nbx_prompt_attn(q, k, v, starts(lens), 1 / math.sqrt(d))
    check(q, k, v, lens, 1 / math.sqrt(d), out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (3, 3), (2, 1), (6, 1), (24, 4), (7, 1), (20, 4), (16, 1), (48, 1), (128, 1),
                                      (32, 32), (256, 1), (192, 1)])
def test_heads(d, h_q, h_kv):
    lens = [70, 200, 9]
    q, k, v = inputs(sum(lens), h_q, h_kv, d, h_q * 7 + h_kv, fused=h_q % 2 == 0)
    out = nbx.nbx_prompt_attn(q, k, v, starts(lens), 1 / math.sqrt(d))
    check(q, k, v, lens, 1 / math.sqrt(d), out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1500, 5000])
def test_long(d, n):
    q, k, v = inputs(n, 4, 2, d, n + d)
    scale = 1 / math.sqrt(d)
    out = nbx.nbx_prompt_attn(q, k, v, starts([n]), scale)
    rows = list(range(0, n, 97)) + [n - 1]
    want, tol = expect(q, k, v, 0, n, scale, rows)
    near(out[rows], want, tol)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 4.0, 1e-30])
def test_scales(d, scale):
    lens = [150, 260]
    q, k, v = inputs(sum(lens), 4, 1, d, d, spread=0.0)
    out = nbx.nbx_prompt_attn(q, k, v, starts(lens), scale)
    check(q, k, v, lens, scale, out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("step", [0.5, -0.5, 30.0, -30.0])
def test_rising_and_falling_scores(d, step):
    """Running maxima that rise with every key, or never after the first."""
    n = 700
    q, k, v = inputs(n, 2, 1, d, 3)
    q.fill_(1.0)
    k.zero_()
    k[:, :, 0] = (torch.arange(n, device=DEV)[:, None] * step / 16).to(torch.bfloat16)
    out = nbx.nbx_prompt_attn(q, k, v, starts([n]), 1.0)
    check(q, k, v, [n], 1.0, out)


def test_far_offsets():
    """Token strides, and rows of q and out, whose offsets pass 2^31 elements."""
    n, stride = 3, (1 << 30) + 64
    base = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(base, (n, 1, 64), (stride, 64, 1))
    x.copy_(torch.randn((n, 1, 64), device=DEV))
    check(x, x, x, [n], 0.125, nbx.nbx_prompt_attn(x, x, x, starts([n]), 0.125))
    del base, x
    n, h = 70_000, 256
    q = torch.empty((n, h, 128), dtype=torch.bfloat16, device=DEV)
    _, k, v = inputs(n, 1, 1, 128, 21)
    lens = [700] * 100
    for lo in (0, 69_300):
        q[lo:lo + 700] = inputs(700, h, 1, 128, lo)[0]
    q[700:69_300] = 1.0
    out = nbx.nbx_prompt_attn(q, k, v, starts(lens), 0.1)
    for lo in (0, 69_300):
        rows = [0, 1, 500, 699]
        want, tol = expect(q, k, v, lo, lo + 700, 0.1, rows)
        near(out[lo:lo + 700][rows], want, tol)


def test_many_short_sequences():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 6, (3000,), generator=g).tolist()
    n = sum(lens)
    q, k, v = inputs(n, 4, 2, 64, 6)
    out = nbx.nbx_prompt_attn(q, k, v, starts(lens), 0.125)
    at = starts(lens).tolist()
    for b in list(range(0, 3000, 61)) + [2998, 2999]:
        if lens[b]:
            near(out[at[b]:at[b + 1]], *expect(q, k, v, at[b], at[b + 1], 0.125))
    # every row is written, and by its own sequence alone
    alone = torch.full_like(out, float("nan"))
    for b in range(0, 3000, 200):
        alone[at[b]:at[b + 1]] = nbx.nbx_prompt_attn(q[at[b]:at[b + 1]], k[at[b]:at[b + 1]], v[at[b]:at[b + 1]],
                                                     starts([lens[b]]), 0.125)
        assert torch.equal(alone[at[b]:at[b + 1]], out[at[b]:at[b + 1]])
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_no_sequence_and_what_lies_in_them(d):
    """Tokens before, between (none) and behind the sequences hold NaN; their rows of the output stay."""
    lens, first = [37, 130, 90], 11
    n = first + sum(lens) + 50
    q, k, v = inputs(n, 4, 2, d, 8)
    for x in (q, k, v):
        x[:first], x[first + sum(lens):] = float("nan"), float("nan")
    out = torch.full((n, 4, d), 9.0, device=DEV, dtype=torch.bfloat16)
    nbx.nbx_prompt_attn(q, k, v, starts(lens, first), 0.1, out=out)
    check(q, k, v, lens, 0.1, out, first)
    assert bool((out[:first] == 9.0).all()) and bool((out[first + sum(lens):] == 9.0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(d, bad, where):
    lens = [100, 300, 20]
    q, k, v = inputs(sum(lens), 4, 2, d, 12, fused=False)
    {"q": q, "k": k, "v": v}[where][100 + 170, 1, 5] = bad
    out = nbx.nbx_prompt_attn(q, k, v, starts(lens), 0.1)
    torch.cuda.synchronize()
    clean = {"q": q, "k": k, "v": v}[where].clone()
    clean[270, 1, 5] = 0.0
    args = {"q": (clean, k, v), "k": (q, clean, v), "v": (q, k, clean)}[where]
    ref = nbx.nbx_prompt_attn(*args, starts(lens), 0.1)
    reached = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    if where == "q":
        reached[270, 1] = True
    else:
        reached[270:400, 2:4] = True
    assert torch.equal(out[~reached], ref[~reached]) or where == "v"   # (rows of a spoilt tile are computed again)
    check(q, k, v, lens, 0.1, out)


def test_scores_of_minus_infinity():
    """Rows whose every score is -inf get 0; later rows, with one finite score, its value."""
    q, k, v = inputs(200, 1, 1, 64, 13, fused=False)
    q.fill_(1.0)
    k[:150, 0, 0] = -float("inf")
    out = nbx.nbx_prompt_attn(q, k, v, starts([200]), 0.1)
    assert bool((out[:150] == 0).all())
    check(q, k, v, [200], 0.1, out)


@pytest.mark.parametrize("start", [[-1, 5, 40], [0, 30, 20, 41], [0, 20, 41], [5, 3, 40]])
def test_bad_bounds(start):
    q, k, v = inputs(40, 2, 1, 64, 14)
    out, status = torch.full((40, 2, 64), 9.0, device=DEV, dtype=torch.bfloat16), ints([0])
    nbx.nbx_prompt_attn(q, k, v, ints(start), 0.1, out=out, status=status)
    assert int(status) == nbx.DEV_BAD_LEN
    held = torch.zeros(40, dtype=torch.bool, device=DEV)
    for a, b in zip(start[:-1], start[1:]):
        if 0 <= a <= b <= 40:
            near(out[a:b], *expect(q, k, v, a, b, 0.1))
            held[a:b] = True
    assert bool((out[~held] == 9.0).all())


def test_the_same_again_and_packed_otherwise():
    lens = [513, 64, 1000, 7]
    q, k, v = inputs(sum(lens), 8, 2, 128, 15)
    one = nbx.nbx_prompt_attn(q, k, v, starts(lens), 0.1)
    assert torch.equal(one, nbx.nbx_prompt_attn(q, k, v, starts(lens), 0.1))
    at = starts(lens).tolist()
    for a, b in zip(at[:-1], at[1:]):
        assert torch.equal(one[a:b], nbx.nbx_prompt_attn(q[a:b], k[a:b], v[a:b], ints([0, b - a]), 0.1))


def test_another_stream_a_replayed_graph_and_two_calls_at_once():
    lens = [200, 90]
    q, k, v = inputs(290, 4, 2, 128, 16)
    q2, k2, v2 = inputs(290, 4, 2, 128, 17)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for s, x in zip(sides * 3, [(q, k, v), (q2, k2, v2)] * 3):
        outs.append(nbx.nbx_prompt_attn(*x, starts(lens), 0.1, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        check(*[(q, k, v), (q2, k2, v2)][i % 2], lens, 0.1, o)
    st, out = starts(lens), torch.empty((290, 4, 128), dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nbx.nbx_prompt_attn(q, k, v, st, 0.1, out=out)
    q.copy_(q2)
    k.copy_(k2)
    v.copy_(v2)
    st.copy_(ints([0, 33, 290]))
    graph.replay()
    check(q, k, v, [33, 257], 0.1, out)


def test_refusals_of_the_binding():
    q, k, v = inputs(20, 4, 2, 64, 18)
    st, call = starts([20]), nbx.nbx_prompt_attn
    for bad in (lambda: call(q.float(), k, v, st, 0.1), lambda: call(q, k[:10], v, st, 0.1), lambda: call(q, k, v[:, :1], st, 0.1),
                lambda: call(q, k, v, st.long(), 0.1), lambda: call(q.transpose(0, 1), k, v, st, 0.1),
                lambda: call(q, k, v, st, 0.1, out=torch.empty_like(q, dtype=torch.float32)),
                lambda: call(q, k, v, st, 0.1, out=q), lambda: call(q, k, v, st[:0], 0.1),
                lambda: call(q, k, v, st, 0.1, status=st[2:]), lambda: call(q, k, v.cpu(), st, 0.1)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(nbx.NbxError):
        call(q[:, :3], k, v, st, 0.1)
    assert call(q[:0], k[:0], v[:0], ints([0, 0]), 0.1).shape == (0, 4, 64)
    call(q, k, v, ints([0]), 0.1)
