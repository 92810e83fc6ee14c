"""The block-scaled decode and the score modifications against their definition in 64 bits (oracle.cache).

Tolerances, from the arithmetic. A weight's relative error is that of its score plus that of 2^x (2^-22).
A score is a sum of d products rounded at most 16 times on its way (8 fused pairs a lane, the pair, a tree
of four, the scale, the block's scale), so it is off by 2^-20 Z, Z = scale |q| |k| a bound on the scores; a
cap or a bias adds less. Sums of weights and of weighted values are fp32, at most 512 terms in a row and 64
splits, hence 2^-14.8 in the worst case. The output is a weighted mean of the values, off by twice the
weights' error times the largest value: max|v| (2^-19 Z + 2^-14). On tensor cores a bf16 window holds P to
2^-17 (two bf16 terms), and an E4M3 window P to 2^-8 (an E4M3 term and an E5M2 one: a rounding to four bits
leaves 2^-4, its rounding to three 2^-4 of that; with the floors of small weights within 2^-8 of the sum) and each element of q to 2^-16 of the vector's largest, so a score to
2^-16 sqrt(d) Z. A bf16 output adds half a step: 2^-8.
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
OUT = {"f32": torch.float32, "bf16": torch.bfloat16}
EDGE_LENS = (0, 1, 15, 16, 17, 100, 255, 256, 257, 513, 1100)


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    nbx.nbx_set_decode_grid_limit(0)
    yield
    nbx.nbx_set_decode_grid_limit(0)


class Case:
    """One decode on both sides. pool: f32, bf16, e4m3 (one scale), block (a scale per T positions)."""

    def __init__(self, pool, q_type, rows, h_q, h_kv, d, P, lens, T=0, seed=0, magnitude=1.0, two=True):
        g = np.random.default_rng(seed)
        self.pool, self.T, self.P, self.d, self.rows, self.h_q = pool, T, P, d, rows, h_q
        self.lens = np.asarray(lens, dtype=np.int32)
        B = len(lens)
        need = [-(-int(n) // P) for n in lens]
        self.num_pages = sum(need) + 2
        self.width = max(1, max(need)) + 1
        ids = g.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((B, self.width), -1, dtype=np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.scale = 1.0 / math.sqrt(d)
        shape = (self.num_pages, h_kv, P, d)
        self.kw, self.scales, self.codes = {}, [None, None], []
        for w in range(2):
            x = (g.standard_normal(shape) * np.exp(0.5 * g.standard_normal(shape[:3] + (1,)))).astype(np.float32)
            x *= magnitude
            if pool == "block":
                s = np.exp2(g.integers(-9, -5, shape[:2] + (P // T,))).astype(np.float32) * np.float32(magnitude)
                if not two:
                    s *= g.uniform(0.6, 1.0, s.shape).astype(np.float32)
                self.scales[w] = s
                x = x / np.repeat(s, T, axis=2)[..., None]
            elif pool == "e4m3":
                self.kw["kv"[w] + "_scale"] = float(np.float32(np.abs(x).max() / 448))
                x = x / self.kw["kv"[w] + "_scale"]
            self.codes.append(of.encode(x, "e4m3" if pool == "block" else pool))
        kind = "e4m3" if pool == "block" else pool
        self.values = [oc.pool_values(c, kind, self.kw.get("kv"[w] + "_scale", 1.0), self.scales[w])
                       for w, c in enumerate(self.codes)]
        # what no sequence holds is NaN on the device
        nan = {"f32": np.float32("nan"), "bf16": np.uint16(0x7FC0), "e4m3": np.uint8(0x7F)}[kind]
        held = np.zeros(shape[:1] + shape[2:3], dtype=bool)
        for b in range(B):
            for j in range(int(lens[b])):
                held[self.table[b, j // P], j % P] = True
        self.dev = []
        for c in self.codes:
            c = c.copy()
            c[np.broadcast_to(~held[:, None, :, None], c.shape)] = nan
            t = torch.from_numpy(c.view(np.int16) if kind == "bf16" else c).to(DEV)
            self.dev.append(t.view(torch.bfloat16) if kind == "bf16" else t)
        q = torch.from_numpy(g.standard_normal((B, rows, h_q, d)).astype(np.float32))
        self.q = q.to(torch.bfloat16 if q_type == "bf16" else torch.float32)

    def call(self, out_type="f32", softcap=0.0, slopes=None, key_begin=None, key_end=None, table=None, **kw):
        i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
        args = dict(softcap=softcap, slopes=None if slopes is None else torch.tensor(slopes, device=DEV),
                    key_begin=i32(key_begin), key_end=i32(key_end), out_dtype=OUT[out_type], **kw)
        most = max(1, int(self.lens.max()))
        t, n = i32(self.table if table is None else table), i32(self.lens)
        if self.pool == "block":
            s = [torch.from_numpy(x).to(DEV) if isinstance(x, np.ndarray) else x for x in self.scales]
            return nbx.nbx_paged_decode_attn_block_scaled(self.q.to(DEV), *self.dev, *s, t, n, most, self.scale, **args)
        return nbx.nbx_paged_decode_attn_modified(self.q.to(DEV), *self.dev, t, n, most, self.scale, **self.kw, **args)

    def tolerance(self, out_type, weight=0.0):
        z = self.scale * float(np.linalg.norm(self.q.float().numpy(), axis=-1).max()) * \
            float(np.linalg.norm(self.values[0], axis=-1).max())
        v = float(np.abs(self.values[1]).max())
        if weight > 2.0 ** -10:
            weight += 2.0 ** -16 * math.sqrt(self.d) * z
        return v * (2.0 ** -19 * z + 2.0 ** -14 + 2 * weight + (2.0 ** -8 if out_type == "bf16" else 0.0))

    def check(self, out_type="f32", weight=0.0, **mod):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = self.call(out_type, status=status, **mod)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        ref = oc.attention(self.q.float().numpy(), *self.values, self.table, self.lens, self.scale, **mod)
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        err = float(np.abs(got - ref).max())
        tol = self.tolerance(out_type, weight)
        assert err <= tol, f"error {err:.3e}, tolerance {tol:.3e}"
        empty = np.all(ref == 0, axis=-1)
        assert np.all(got[empty] == 0)
        return out


def slopes_for(h):
    return [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]


def ranges(kind, lens, rows, seed=0):
    """(key_begin, key_end) [B, rows]."""
    n = np.asarray(lens, dtype=np.int64)[:, None]
    p = n - rows + np.arange(rows)[None, :]
    if kind == "documents":
        return np.maximum(p, 0) // 100 * 100, p + 1
    if kind == "prefix":
        return None, np.maximum(p + 1, 70)
    if kind == "window":
        return np.maximum(0, p + 1 - 37), None
    g = np.random.default_rng(seed)
    lo = g.integers(-5, np.maximum(n, 1) + 5, p.shape)        # anything: empty rows, ends before starts, outside
    return lo, lo + g.integers(-20, 400, p.shape)


SIMT = [("f32", "f32", 1, 4, 2, 64, 16, 0), ("bf16", "bf16", 1, 32, 8, 128, 16, 0), ("bf16", "f32", 3, 12, 4, 256, 64, 0),
        ("e4m3", "bf16", 1, 8, 8, 128, 32, 0), ("e4m3", "f32", 5, 6, 2, 64, 16, 0), ("block", "bf16", 1, 32, 8, 128, 16, 16),
        ("block", "f32", 2, 6, 1, 256, 64, 32), ("block", "bf16", 7, 8, 2, 64, 128, 128), ("f32", "bf16", 4, 5, 1, 128, 512, 0),
        ("block", "bf16", 1, 7, 1, 128, 48, 16)]
MODS = [dict(), dict(softcap=2.0), dict(slopes=True), dict(mask="documents"), dict(mask="prefix"), dict(mask="window"),
        dict(mask="random", softcap=5.0, slopes=True)]


def made(mod, lens, rows, h_q):
    m = {k: v for k, v in mod.items() if k == "softcap"}
    if "slopes" in mod:
        m["slopes"] = np.float32(slopes_for(h_q)).tolist()
    if "mask" in mod:
        m["key_begin"], m["key_end"] = ranges(mod["mask"], lens, rows)
    return m


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(str(v) for v in m.values()) or "plain")
@pytest.mark.parametrize("pool,q_type,rows,h_q,h_kv,d,P,T", SIMT)
def test_single_rows_and_short_windows(pool, q_type, rows, h_q, h_kv, d, P, T, mod):
    c = Case(pool, q_type, rows, h_q, h_kv, d, P, EDGE_LENS, T, seed=1, two=(rows == 1))
    for out_type in ("f32", "bf16"):
        c.check(out_type, **made(mod, EDGE_LENS, rows, h_q))


def test_a_cap_on_large_scores():
    # scores up to a hundred times the cap, and far under it
    for magnitude in (100.0, 1e-3):
        c = Case("bf16", "f32", 1, 8, 2, 128, 16, (1, 40, 700), seed=2, magnitude=magnitude)
        out = c.call(softcap=30.0)
        ref = oc.attention(c.q.numpy(), *c.values, c.table, c.lens, c.scale, softcap=30.0)
        # capped scores are off by at most 30 * 2^-22 (tanhf) and what is left of the score's own error there,
        # s 2^-20 tanh'(s / 30) <= 30 * 2^-20
        tol = float(np.abs(c.values[1]).max()) * (2 * 30 * 2.0 ** -19 + 2.0 ** -14)
        assert np.abs(out.double().cpu().numpy() - ref).max() <= tol


def test_slopes_of_any_sign_and_size():
    c = Case("bf16", "bf16", 2, 8, 2, 128, 16, (3, 600, 1500), seed=3)
    for s in (0.0, -0.01, 1e4, 1e-8):
        c.check(slopes=[s] * 8)
    c.check(slopes=[1e30] * 8)          # all weight on the row's own position


def test_many_vectors_of_a_pool_without_tensor_core_windows():
    # windows of 64 and more vectors that the window kernel does not take: pages of 16, d 64, fp32 queries
    for pool, q_type, rows, h_q, h_kv, d, P, T in (("block", "bf16", 40, 8, 2, 128, 16, 16), ("e4m3", "f32", 70, 4, 1, 256, 64, 0),
                                                   ("bf16", "bf16", 130, 3, 1, 64, 64, 0), ("bf16", "f32", 33, 4, 2, 128, 64, 0)):
        c = Case(pool, q_type, rows, h_q, h_kv, d, P, (3, 200, 777), T, seed=16)
        for mod in (MODS[0], MODS[3], MODS[6]):
            c.check("f32", **made(mod, c.lens, rows, h_q))


def test_a_nan_value_seen_by_some_vectors_of_a_tile():
    # the key-by-key path of a tile: a NaN (and, in bf16, an infinity) that two of three rows see
    for pool, T in (("e4m3", 0), ("block", 16), ("bf16", 0)):
        for d in (64, 128, 256):
            c = Case(pool, "bf16", 3, 4, 2, d, 16, (100,), T, seed=17)
            lo = np.array([[0, 20, 40]])
            ref = oc.attention(c.q.float().numpy(), *c.values, c.table, c.lens, c.scale, key_begin=lo)
            c.dev[1][c.table[0, 1], :, 9, 5] = 0x7F if pool != "bf16" else float("nan")      # position 25
            if pool == "bf16":
                c.dev[1][c.table[0, 0], :, 3, 6] = float("-inf")                             # position 3
            out = c.call(key_begin=lo).double().cpu().numpy()
            assert np.all(np.isnan(out[0, :2, :, 5])) and np.all(np.isfinite(out[0, 2]))
            if pool == "bf16":
                assert np.all(np.isneginf(out[0, 0, :, 6])) and np.all(np.isfinite(out[0, 1, :, 6]))
            keep = np.ones(d, dtype=bool)
            keep[5:7] = False
            assert np.abs(out[0][:, :, keep] - ref[0][:, :, keep]).max() <= c.tolerance("f32")


def test_queries_of_any_size():
    # the E4M3 kernels scale a query vector by a power of two: tiny, huge, zero, with elements far apart
    for q_type in ("bf16", "f32"):
        c = Case("block", q_type, 1, 8, 2, 128, 16, (200, 90), 16, seed=18)
        q = c.q.float()
        q[0, 0, 0] = 0.0
        q[0, 0, 1] *= 1e-30
        q[0, 0, 2] *= 1e-3
        q[0, 0, 3, 5] = 300.0
        q[1, 0, 4] *= torch.logspace(-12, 0, 128)
        q[1, 0, 5] = float("nan")
        q[1, 0, 6, 7] = float("inf")
        c.q = q.to(c.q.dtype)
        out = c.call().double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            ref = oc.attention(c.q.float().numpy(), *c.values, c.table, c.lens, c.scale)
        assert np.all(np.isnan(out[1, 0, 5])) and np.all(np.isnan(out[1, 0, 6]) | np.isfinite(out[1, 0, 6]))
        c.q[1, 0, 5:7] = 0.0
        c.q[0, 0, 3] = 0.0          # (its scores are large: left out of the tolerance's bound)
        out[1, 0, 5:7] = ref[1, 0, 5:7] = out[0, 0, 3] = ref[0, 0, 3] = 0.0
        assert np.abs(out - ref).max() <= c.tolerance("f32")


def test_pages_no_row_sees_may_be_gone():
    # a window of 37 keys: the pages before it are -1, as a serving loop frees them; and out of the pool
    for pool, T in (("bf16", 0), ("block", 16)):
        c = Case(pool, "bf16", 3, 8, 2, 128, 16, (600, 1300, 40), T, seed=4)
        lo, _ = ranges("window", c.lens, 3)
        whole = c.call(key_begin=lo)
        t = c.table.copy()
        for b in range(3):
            t[b, : int(lo[b].min()) // 16] = -1 if b else 10 ** 6
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = c.call(key_begin=lo, table=t, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and torch.equal(out, whole)


def test_nan_and_infinity_outside_the_ranges_stay_outside():
    for pool in ("f32", "bf16"):
        c = Case(pool, "f32", 4, 4, 1, 64, 16, (300,), seed=5)
        lo, hi = np.array([[50, 60, 70, 0]]), np.array([[100, 61, 200, 0]])
        ref = oc.attention(c.q.numpy(), *c.values, c.table, c.lens, c.scale, key_begin=lo, key_end=hi)
        for j, bad in ((49, "nan"), (200, "inf"), (10, "-inf"), (299, "nan")):
            for w in range(2):
                c.dev[w][c.table[0, j // 16], :, j % 16] = float(bad)
        out = c.call(key_begin=lo, key_end=hi).double().cpu().numpy()
        assert np.abs(out - ref).max() <= c.tolerance("f32")
        # a NaN that is seen reaches the rows that see it, and no other
        c.dev[0][c.table[0, 60 // 16], :, 60 % 16] = float("nan")
        out = c.call(key_begin=lo, key_end=hi).cpu().numpy()
        assert np.all(np.isnan(out[0, :2])) and np.all(np.isfinite(out[0, 2:]))


def test_without_modifications_it_is_the_plain_decode():
    c = Case("bf16", "bf16", 1, 32, 8, 128, 16, (5, 900, 2000), seed=6)
    i32 = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    plain = nbx.nbx_paged_decode_attn(c.q.to(DEV), *c.dev, i32(c.table), i32(c.lens), 2000, c.scale)
    assert torch.equal(plain, c.call())
    # slopes of 0 and a cap far above the scores: other kernels, the same numbers
    for other in (c.call(slopes=[0.0] * 32), c.call(softcap=1e6), c.call("bf16")):
        err = float((plain.double() - other.double()).abs().max())
        assert err <= c.tolerance("bf16" if other.dtype == torch.bfloat16 else "f32") + c.tolerance("f32")


def test_block_scales_of_one_are_the_plain_decode():
    c = Case("block", "bf16", 1, 32, 8, 128, 16, (5, 900, 2000), 16, seed=7)
    c.scales = [np.ones_like(s) for s in c.scales]
    c.values = [oc.pool_values(x, "e4m3", scales=s) for x, s in zip(c.codes, c.scales)]
    i32 = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    plain = nbx.nbx_paged_decode_attn(c.q.to(DEV), *c.dev, i32(c.table), i32(c.lens), 2000, c.scale)
    assert float((plain - c.call()).abs().max()) <= 2 * c.tolerance("f32")


def test_scales_at_the_ends_of_their_range():
    # a block of tiny values beside a block of large ones: the weights of both count
    c = Case("block", "f32", 1, 4, 1, 128, 16, (64, 33), 16, seed=8)
    g = np.random.default_rng(8)
    c.scales[1] = np.where(g.random(c.scales[1].shape) < 0.5, np.float32(2.0 ** -48), np.float32(2.0 ** 48))
    c.values[1] = oc.pool_values(c.codes[1], "e4m3", scales=c.scales[1])
    out = c.call().double().cpu().numpy()
    ref = oc.attention(c.q.numpy(), *c.values, c.table, c.lens, c.scale)
    assert np.abs(out - ref).max() <= c.tolerance("f32")


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** -49, 2.0 ** 49])
def test_a_bad_scale_sets_its_bit_and_its_block_is_skipped(bad):
    c = Case("block", "bf16", 1, 8, 2, 128, 32, (200, 90), 16, seed=9)
    page = int(c.table[0, 2])
    for w in range(2):
        c.scales[w] = torch.from_numpy(c.scales[w]).to(DEV)
        good = c.scales[w].clone()
        c.scales[w][page, 1, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = c.call(status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == nbx.DEV_BAD_SCALE
        c.scales[w] = good
        # positions 80..95 of KV head 1 of sequence 0 are as if they were not there
        keep = [j for j in range(200) if not 80 <= j < 96]
        K, V = (x[c.table[0, :7].astype(int), 1].reshape(-1, 128)[keep] for x in c.values)
        s = c.scale * (c.q[0, 0, 4:].double().numpy() @ K.T)
        e = np.exp(s - s.max(-1, keepdims=True))
        ref = e @ V / e.sum(-1, keepdims=True)
        assert np.abs(out[0, 0, 4:].double().cpu().numpy() - ref).max() <= c.tolerance("f32")
        assert torch.equal(out[1], c.call()[1])


def test_bad_pages_and_lengths_are_reported():
    c = Case("block", "bf16", 1, 8, 2, 128, 16, (200, 90), 16, seed=10)
    t = c.table.copy()
    t[0, 3] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.call(table=t, status=status, slopes=[0.1] * 8)
    torch.cuda.synchronize()
    assert int(status.item()) == nbx.DEV_BAD_PAGE and bool(torch.isfinite(out).all())
    n = c.lens.copy()
    c.lens = np.array([-1, 90], dtype=np.int32)
    status.zero_()
    out = c.call(status=status, key_begin=np.zeros((2, 1)))
    torch.cuda.synchronize()
    assert int(status.item()) == nbx.DEV_BAD_LEN and bool((out[0] == 0).all())
    c.lens = n


# ------------------------------------------------------------------------------------------------ tensor cores
# rows x group of 64 and more, bf16 q, d 128 or 256, pages of whole 64-position tiles
TENSOR = [("bf16", 16, 24, 4, 256, 64, 0), ("bf16", 8, 32, 4, 128, 128, 0), ("bf16", 70, 12, 4, 128, 64, 0),
          ("e4m3", 16, 24, 4, 256, 64, 0), ("e4m3", 33, 8, 2, 128, 192, 0), ("block", 16, 24, 4, 256, 64, 64),
          ("block", 8, 32, 4, 128, 64, 16), ("block", 40, 4, 1, 128, 128, 128), ("block", 130, 2, 2, 256, 128, 32),
          ("bf16", 128, 2, 1, 128, 512, 0)]
WINDOW_LENS = (0, 1, 17, 63, 64, 65, 129, 300, 513, 1100)
P_WEIGHT = {"bf16": 2.0 ** -17, "e4m3": 2.0 ** -7, "block": 2.0 ** -7}


def on_tensor_cores(c, out_type):
    kind = nbx.NBX_BF16 if c.pool == "bf16" else nbx.NBX_E4M3
    h_kv = c.dev[0].shape[1]
    return nbx.nbx_paged_decode_modified_partial_kernel(nbx.dtype_code(c.q), kind, nbx.NBX_BF16 if out_type == "bf16" else
                                                        nbx.NBX_F32, c.rows, c.h_q, h_kv, c.d, c.num_pages,
                                                        c.P) in (nbx.PARTIAL_TCGEN05, nbx.PARTIAL_TCGEN05_FP8)


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(str(v) for v in m.values()) or "plain")
@pytest.mark.parametrize("pool,rows,h_q,h_kv,d,P,T", TENSOR)
def test_windows_on_tensor_cores(pool, rows, h_q, h_kv, d, P, T, mod):
    c = Case(pool, "bf16", rows, h_q, h_kv, d, P, WINDOW_LENS, T, seed=20, two=(rows != 8))
    assert on_tensor_cores(c, "bf16")
    c.check("bf16", weight=P_WEIGHT[pool], **made(mod, WINDOW_LENS, rows, h_q))
    if pool == "bf16":
        c.check("f32", weight=P_WEIGHT[pool], **made(mod, WINDOW_LENS, rows, h_q))
    else:
        assert not on_tensor_cores(c, "f32")


def test_fp8_windows_with_an_fp32_output_keep_fp32_weights():
    c = Case("block", "bf16", 16, 24, 4, 256, 64, (5, 400), 32, seed=21)
    c.check("f32", softcap=5.0)


@pytest.mark.parametrize("pool,T", [("bf16", 0), ("e4m3", 0), ("block", 16)])
def test_one_cta_runs_every_unit_of_a_masked_window(pool, T):
    # units of one tile, of many, and of none that any row sees, one after another on one CTA
    c = Case(pool, "bf16", 64, 8, 2, 128, 64, (2000, 70, 900, 0, 64), T, seed=22)
    mod = made(dict(mask="random", softcap=4.0, slopes=True), c.lens, 64, 8)
    ref = c.call("bf16", **mod)
    for limit in (1, 3):
        nbx.nbx_set_decode_grid_limit(limit)
        out = c.call("bf16", **mod)
        nbx.nbx_set_decode_grid_limit(0)
        assert torch.equal(out, ref)
    c.check("bf16", weight=P_WEIGHT[pool], **mod)


def test_windows_with_gone_pages():
    for pool, T in (("bf16", 0), ("block", 64)):
        c = Case(pool, "bf16", 16, 16, 2, 128, 64, (1600, 2300, 40), T, seed=23)
        lo, _ = ranges("window", c.lens, 16)
        whole = c.call("bf16", key_begin=lo)
        t = c.table.copy()
        for b in range(3):
            t[b, : int(lo[b].min()) // 64] = -1
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = c.call("bf16", key_begin=lo, table=t, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and torch.equal(out, whole)


@pytest.mark.parametrize("lens", [(300,), (3000,)])       # one split, and several
@pytest.mark.parametrize("pool,T", [("bf16", 0), ("e4m3", 0), ("block", 16)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(pool, T, lens):
    n, rows = lens[0], 64
    c = Case(pool, "bf16", rows, 4, 1, 128, 64, lens, T, seed=24)
    lo = np.zeros((1, rows), dtype=np.int64)
    lo[0, 32:] = 100                              # rows 32.. do not see position 50
    lo[0, 60] = n                                 # row 60 sees nothing
    ref = oc.attention(c.q.float().numpy(), *c.values, c.table, c.lens, c.scale, key_begin=lo, softcap=3.0)
    at = (c.table[0, 0], slice(None), 50)
    for w in range(2):
        c.dev[w][at] = 0x7F if pool != "bf16" else float("nan")
    last = (c.table[0, (n - 1) // 64], slice(None), (n - 1) % 64)    # seen by the last row alone
    if pool == "bf16":
        c.dev[1][last] = float("inf")
    out = c.call("bf16", key_begin=lo, softcap=3.0).double().cpu().numpy()
    assert np.all(np.isnan(out[0, :32]))
    stop = rows - 1 if pool == "bf16" else rows
    assert np.abs(out[0, 32:stop] - ref[0, 32:stop]).max() <= c.tolerance("bf16", P_WEIGHT[pool])
    assert np.all(out[0, 60] == 0)
    if pool == "bf16":
        assert np.all(np.isposinf(out[0, -1]))


def test_scales_far_apart_in_a_window():
    # a sink: a block of nearly zero values that takes most of the weight beside blocks of ordinary ones
    for small in (2.0 ** -20, 2.0 ** -48):
        c = Case("block", "bf16", 64, 4, 1, 128, 64, (700,), 16, seed=25)
        first = (int(c.table[0, 0]), 0, 0)
        c.scales[1] = c.scales[1].copy()
        c.scales[1][first] = small
        c.values[1] = oc.pool_values(c.codes[1], "e4m3", scales=c.scales[1])
        k = c.values[0][first[0], 0, :16]
        c.q = (c.q + 3.0 * torch.from_numpy(k.mean(0)).float()).to(torch.bfloat16)
        c.check("bf16", weight=P_WEIGHT["block"])
        c.check("bf16", weight=P_WEIGHT["block"], slopes=[0.01] * 4)


def test_a_bad_scale_in_a_window():
    c = Case("block", "bf16", 64, 4, 1, 128, 64, (700,), 16, seed=26)
    page = int(c.table[0, 3])
    s = c.scales[1].copy()
    s[page, 0, 2] = float("nan")
    c.scales[1] = s
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.call("bf16", status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == nbx.DEV_BAD_SCALE
    keep = [j for j in range(700) if not 3 * 64 + 32 <= j < 3 * 64 + 48]
    vals = [x[c.table[0, :11].astype(int), 0].reshape(-1, 128) for x in c.values]
    for r in (0, 33, 63):
        seen = [j for j in keep if j <= 700 - 64 + r]
        z = c.scale * (c.q[0, r].double().numpy() @ vals[0][seen].T)
        e = np.exp(z - z.max(-1, keepdims=True))
        ref = e @ vals[1][seen] / e.sum(-1, keepdims=True)
        c.values[1] = np.nan_to_num(c.values[1])
        assert np.abs(out[0, r].double().cpu().numpy() - ref).max() <= c.tolerance("bf16", P_WEIGHT["block"])


def test_a_wait_that_runs_out_in_a_modified_window_returns_with_its_bit():
    for pool, T in (("bf16", 0), ("block", 64)):
        c = Case(pool, "bf16", 16, 24, 4, 256, 64, (1500, 900), T, seed=27)
        nbx.nbx_set_decode_wait_test(200_000, 20_000_000)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        c.call("bf16", status=status, softcap=4.0)
        torch.cuda.synchronize()
        nbx.nbx_set_decode_wait_test(0, 0)
        assert int(status.item()) & nbx.DEV_TIMEOUT
        c.check("bf16", weight=P_WEIGHT[pool], softcap=4.0)


@pytest.mark.parametrize("pool,T", [("bf16", 0), ("block", 16)])
def test_grid_size_and_page_ids_do_not_change_bits(pool, T):
    c = Case(pool, "bf16", 2, 16, 4, 128, 16, (900, 3, 2000, 0, 700), T, seed=11)
    mod = made(dict(mask="documents", softcap=3.0, slopes=True), c.lens, 2, 16)
    ref = c.call(**mod)
    for limit in (1, 7, 100):
        nbx.nbx_set_decode_grid_limit(limit)
        out = c.call(**mod)
        nbx.nbx_set_decode_grid_limit(0)
        assert torch.equal(out, ref)
    perm = np.random.default_rng(12).permutation(c.num_pages)
    inv = torch.from_numpy(np.argsort(perm)).to(DEV)
    c.dev = [t[inv] for t in c.dev]
    if T:
        c.scales = [s[np.argsort(perm)] for s in c.scales]
    t = np.where(c.table >= 0, perm[np.maximum(c.table, 0)], c.table)
    assert torch.equal(c.call(table=t, **mod), ref)


def test_more_sequences_than_the_plan_sorts():
    B = 2100
    lens = np.random.default_rng(13).integers(0, 40, B)
    c = Case("block", "bf16", 1, 2, 1, 64, 16, lens, 16, seed=13)
    c.check(**made(dict(mask="window", softcap=3.0), lens, 1, 2))


def test_two_streams_and_a_replayed_graph():
    c = Case("block", "bf16", 1, 8, 2, 128, 16, (900, 3, 2000), 16, seed=14)
    i32 = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    need = nbx.nbx_paged_decode_modified_workspace_bytes(3, 1, 8, 2, 128, 2000)
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.zeros(c.q.shape, device=DEV) for _ in range(2)]
    s = [torch.from_numpy(x).to(DEV) for x in c.scales]
    q, t, n = c.q.to(DEV), i32(c.table), i32(c.lens)
    run = lambda i, q: nbx.nbx_paged_decode_attn_block_scaled(q, *c.dev, *s, t, n, 2000, c.scale, softcap=4.0 + i,  # noqa: E731
                                                             out=outs[i], workspace=ws[i])
    ref = [run(i, q).clone() for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):         # both at once
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                run(i, q)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    q2 = q.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(0, q2)
    q2.copy_(torch.randn_like(q2.float()).to(q2.dtype))
    g.replay()
    torch.cuda.synchronize()
    got = outs[0].clone()
    assert torch.equal(got, run(0, q2))


def test_refusals_of_the_bindings():
    c = Case("block", "bf16", 1, 8, 2, 128, 32, (200, 90), 16, seed=15)
    with pytest.raises(ValueError):
        c.call(key_begin=np.zeros((2, 2)))
    with pytest.raises(ValueError):
        c.call(slopes=[0.1] * 7)
    with pytest.raises(ValueError):
        c.call(out=torch.empty((2, 1, 8, 64), device=DEV))
    with pytest.raises(nbx.NbxError):
        c.call(softcap=-1.0)
    with pytest.raises(nbx.NbxError):
        c.call(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        nbx.nbx_paged_decode_attn_block_scaled(c.q.to(DEV), *c.dev, *[torch.from_numpy(x).to(DEV) for x in c.scales],
                                               torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.lens).to(DEV), 200,
                                               c.scale, out_dtype=torch.float16)
    half = [s[:, :, :1].copy() for s in c.scales]
    c.scales = [half[0], c.scales[1]]
    with pytest.raises(ValueError):
        c.call()


def test_large_bf16_values_stay_finite():
    # values of 1e36 under weights held up to 2^8 of their row's largest: no sum leaves fp32's range
    c = Case("bf16", "bf16", 1, 8, 2, 128, 16, (300, 33), 0, seed=77)
    v = c.dev[1].float().nan_to_num(0.0).clamp(-1.0, 1.0) * 1e36
    c.dev[1] = v.to(torch.bfloat16)
    c.values = [c.values[0], c.dev[1].double().cpu().numpy() * c.kw.get("v_scale", 1.0)]
    c.check(softcap=3.0)


@pytest.mark.parametrize("pool,rows,h_q,h_kv,batch,longest", [
    ("bf16", 128, 16, 4, 10, 700),       # 160 units, dealt out by their keys
    ("block", 128, 16, 4, 10, 700),
    ("bf16", 32, 16, 1, 100, 150),       # 400 M tiles: more than the plan's threads, fewer than it sorts
    ("bf16", 32, 16, 1, 131, 150),       # more M tiles than the plan sorts
])
def test_windows_of_many_units_over_key_ranges(pool, rows, h_q, h_kv, batch, longest):
    """More work units than SMs, of uneven length: each is done once, on a full grid and on 7 CTAs."""
    lens = np.random.default_rng(5).integers(rows, longest, batch)
    lens[3] = 0
    c = Case(pool, "bf16", rows, h_q, h_kv, 128, 64, lens, 64 if pool == "block" else 0, seed=88)
    for mask in ("documents", "random"):
        mod = made(dict(mask=mask), c.lens, rows, h_q)
        out = c.check("bf16", P_WEIGHT[pool], **mod)
        nbx.nbx_set_decode_grid_limit(7)
        try:
            assert torch.equal(c.call("bf16", **mod), out)
        finally:
            nbx.nbx_set_decode_grid_limit(0)


@pytest.mark.parametrize("batch,rows", [(700, 1), (2048, 1), (2049, 1), (300, 3), (70, 40)])
@pytest.mark.parametrize("pool", ["f32", "bf16"])
def test_key_ranges_of_large_batches(pool, batch, rows):
    lens = np.random.default_rng(batch).integers(0, 60, batch)
    c = Case(pool, "f32" if pool == "f32" else "bf16", rows, 2, 1, 64, 16, lens, seed=89)
    c.check(**made(dict(mask="random"), c.lens, rows, 2))
    c.check(**made(dict(mask="window", softcap=4.0), c.lens, rows, 2))


@pytest.mark.parametrize("pool,rows,h_q,h_kv,d,P,T", [
    ("bf16", 12, 8, 2, 128, 64, 0), ("block", 15, 4, 1, 128, 64, 64), ("e4m3", 10, 8, 2, 128, 128, 0),
    ("bf16", 6, 12, 2, 256, 64, 0), ("block", 8, 4, 1, 256, 64, 16), ("e4m3", 11, 6, 2, 256, 64, 0)])
def test_small_windows_with_a_bf16_output(pool, rows, h_q, h_kv, d, P, T):
    """Windows of 32 to 63 query vectors of a KV head: on the tensor cores for a bf16 output alone."""
    c = Case(pool, "bf16", rows, h_q, h_kv, d, P, (0, 1, 63, 200, 1500), T, seed=90)
    assert on_tensor_cores(c, "bf16") and not on_tensor_cores(c, "f32")
    for mod in (MODS[0], MODS[1], MODS[5], MODS[6]):
        c.check("bf16", P_WEIGHT[pool], **made(mod, c.lens, rows, h_q))
        c.check("f32", **made(mod, c.lens, rows, h_q))
