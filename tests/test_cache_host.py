"""The block-scaled append and the page calls without a GPU: what they refuse on the host before any CUDA
call, and their definitions (oracle.cache) on cases small enough to read."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.formats as of
import paged_split_kv_append_gb300 as nbx

NULL = None
FAKE = ctypes.c_void_p(0x10000)          # a 16-byte aligned address that is never dereferenced
FAKE_ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    nbx.build()
    return nbx.lib()


def call(f, defaults, **kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return f(*a.values())


APPEND = dict(new_k=FAKE, new_v=FAKE, new_dtype=1, n_tok=4, h_kv=2, d=128, k_pool=FAKE, v_pool=FAKE, ks=FAKE, vs=FAKE,
              block=16, num_pages=8, page_tokens=32, bt=FAKE, max_pages=4, batch=2, lens=FAKE, start=FAKE, status=NULL,
              stream=NULL)


@pytest.mark.parametrize("want,kw", [
    (0, dict(n_tok=0)), (0, dict(batch=0)), (-1, dict(new_k=NULL)), (-1, dict(vs=NULL)), (-1, dict(bt=NULL)),
    (-1, dict(start=NULL)), (-2, dict(d=96)), (-2, dict(d=512)), (-2, dict(h_kv=0)), (-2, dict(n_tok=-1)),
    (-2, dict(batch=-1)), (-2, dict(max_pages=0)), (-2, dict(num_pages=0)), (-3, dict(new_dtype=2)),
    (-3, dict(new_dtype=9)), (-4, dict(block=0)), (-4, dict(block=8)), (-4, dict(block=48, page_tokens=96)),
    (-4, dict(block=64)), (-4, dict(block=256, page_tokens=256)), (-7, dict(k_pool=FAKE_ODD)),
    (-7, dict(new_v=FAKE_ODD))])
def test_block_append_refusals(lib, want, kw):
    assert call(lib.nbx_paged_kv_append_block_scaled, APPEND, **kw) == want


POOLS = dict(k_pool=FAKE, v_pool=FAKE, pool_dtype=1, num_pages=8, h_kv=2, page_tokens=32, d=128, ks=NULL, vs=NULL, block=0)
COPY = dict(moves=FAKE, n=FAKE, max_moves=3, **POOLS, status=NULL, stream=NULL)
FORK = dict(bt=FAKE, max_pages=4, lens=FAKE, batch=5, src=FAKE, dst=FAKE, n_fork=2, **POOLS, moves=FAKE, n=FAKE, ws=FAKE,
            ws_bytes=1 << 20, status=NULL, stream=NULL)
COMPACT = dict(bt=FAKE, new_bt=FAKE, max_pages=4, lens=FAKE, batch=5, **POOLS, moves=FAKE, max_moves=4, counts=FAKE,
               ws=FAKE, ws_bytes=1 << 20, status=NULL, stream=NULL)
BAD_POOLS = [(-1, dict(v_pool=NULL)), (-2, dict(num_pages=0)), (-2, dict(page_tokens=0)), (-2, dict(d=8)),
             (-2, dict(d=72)), (-2, dict(d=2048)), (-2, dict(h_kv=0)), (-2, dict(page_tokens=1 << 24)),
             (-3, dict(pool_dtype=7)), (-3, dict(ks=FAKE, vs=FAKE, block=16)),
             (-4, dict(pool_dtype=2, ks=FAKE, vs=FAKE, block=24)), (-1, dict(pool_dtype=2, ks=FAKE, block=16)),
             (-7, dict(k_pool=FAKE_ODD))]


@pytest.mark.parametrize("want,kw", BAD_POOLS + [(0, dict(max_moves=0)), (-2, dict(max_moves=-1)), (-1, dict(moves=NULL)),
                                                 (-1, dict(n=NULL)), (-1, dict(k_pool=NULL, v_pool=NULL))])
def test_copy_refusals(lib, want, kw):
    assert call(lib.nbx_paged_kv_copy_pages, COPY, **kw) == want


@pytest.mark.parametrize("want,kw", BAD_POOLS + [
    (0, dict(n_fork=0)), (0, dict(batch=0)), (-2, dict(n_fork=-1)), (-2, dict(batch=-1)), (-2, dict(max_pages=0)),
    (-2, dict(batch=1 << 20, max_pages=1 << 12)), (-1, dict(bt=NULL)), (-1, dict(src=NULL)), (-1, dict(moves=NULL)),
    (-1, dict(n=NULL)), (-1, dict(ws=NULL)), (-7, dict(ws=ctypes.c_void_p(0x10010))), (-5, dict(ws_bytes=100))])
def test_fork_refusals(lib, want, kw):
    assert call(lib.nbx_paged_kv_fork, FORK, **kw) == want


@pytest.mark.parametrize("want,kw", BAD_POOLS + [
    (0, dict(batch=0)), (-2, dict(max_moves=3)), (-2, dict(num_pages=(1 << 30) + 1, max_moves=1 << 30)),
    (-1, dict(new_bt=NULL)), (-1, dict(counts=NULL)), (-1, dict(moves=NULL)), (-1, dict(lens=NULL)),
    (-7, dict(ws=ctypes.c_void_p(0x10010))), (-5, dict(ws_bytes=100))])
def test_compact_refusals(lib, want, kw):
    assert call(lib.nbx_paged_kv_compact, COMPACT, **kw) == want


SIZES = dict(q=FAKE, q_dtype=1, batch=2, rows=1, h_q=8, d=128, k_pool=FAKE, v_pool=FAKE)
TAIL = dict(softcap=0.0, slopes=NULL, kb=NULL, ke=NULL, out=FAKE, out_dtype=0, ws=FAKE, ws_bytes=1 << 30, status=NULL,
            stream=NULL)
MODIFIED = dict(**SIZES, pool_dtype=1, num_pages=100, h_kv=2, page_tokens=32, bt=FAKE, max_pages=10, lens=FAKE,
                max_seq_len=160, scale=0.1, k_scale=1.0, v_scale=1.0, **TAIL)
BLOCK = dict(**SIZES, ks=FAKE, vs=FAKE, block=16, num_pages=100, h_kv=2, page_tokens=32, bt=FAKE, max_pages=10, lens=FAKE,
             max_seq_len=160, scale=0.1, **TAIL)
BAD_DECODE = [(0, dict(batch=0)), (-1, dict(q=NULL)), (-1, dict(out=NULL)), (-1, dict(bt=NULL)), (-1, dict(ws=NULL)),
              (-2, dict(h_q=9)), (-2, dict(d=96)), (-2, dict(rows=0)), (-2, dict(max_seq_len=321)), (-3, dict(q_dtype=2)),
              (-3, dict(out_dtype=2)), (-4, dict(page_tokens=40, max_seq_len=100)), (-5, dict(ws_bytes=1000)),
              (-7, dict(out=FAKE_ODD)), (-7, dict(q=FAKE_ODD)), (-7, dict(ws=ctypes.c_void_p(0x10010))),
              (-8, dict(scale=float("nan"))), (-8, dict(softcap=-1.0)), (-8, dict(softcap=float("inf"))),
              (-8, dict(softcap=float("nan"))), (-8, dict(softcap=1e-40))]


@pytest.mark.parametrize("want,kw", BAD_DECODE + [(-3, dict(pool_dtype=7)), (-8, dict(v_scale=0.0))])
def test_modified_decode_refusals(lib, want, kw):
    assert call(lib.nbx_paged_decode_attn_modified, MODIFIED, **kw) == want


@pytest.mark.parametrize("want,kw", BAD_DECODE + [(-1, dict(ks=NULL)), (-4, dict(block=0)), (-4, dict(block=24)),
                                                  (-4, dict(block=64))])
def test_block_scaled_decode_refusals(lib, want, kw):
    assert call(lib.nbx_paged_decode_attn_block_scaled, BLOCK, **kw) == want


def test_modified_decode_workspace(lib):
    f = lib.nbx_paged_decode_modified_workspace_bytes
    assert f(2, 1, 8, 3, 128, 100) == 0
    n = f(2, 1, 8, 2, 128, 160)
    assert n >= lib.nbx_paged_decode_workspace_bytes(2, 1, 8, 2, 128, 160)
    assert call(lib.nbx_paged_decode_attn_modified, MODIFIED, ws_bytes=n - 1) == -5


def test_page_workspaces(lib):
    assert lib.nbx_paged_kv_fork_workspace_bytes(-1, 4, 2, 8) == 0
    assert lib.nbx_paged_kv_fork_workspace_bytes(5, 4, 2, 0) == 0
    assert lib.nbx_paged_kv_compact_workspace_bytes(0) == 0
    n = lib.nbx_paged_kv_fork_workspace_bytes(5, 4, 2, 8)
    assert call(lib.nbx_paged_kv_fork, FORK, ws_bytes=n - 1) == -5
    n = lib.nbx_paged_kv_compact_workspace_bytes(8)
    assert call(lib.nbx_paged_kv_compact, COMPACT, ws_bytes=n - 1) == -5


def test_bindings_refuse_host_tensors():
    t = torch.zeros((4, 2, 16, 64))
    i = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        nbx.nbx_paged_kv_fork(i, i[0], i[0], i[0], t, t)
    with pytest.raises(ValueError):
        nbx.nbx_paged_kv_compact(i, i[0], t, t)
    with pytest.raises(ValueError):
        nbx.nbx_paged_kv_copy_pages(i, i[0], t, t)
    with pytest.raises(ValueError):
        nbx.nbx_paged_kv_append_block_scaled(t[0], t[0], t, t, t, t, i, i[0], i[0])


# ------------------------------------------------------------------------------------------------ definitions
def test_block_scale_is_the_smallest_power_that_holds():
    assert oc.block_scale(448.0) == 1.0 and oc.block_scale(448.1) == 2.0 and oc.block_scale(1.75) == 2.0 ** -8
    assert oc.block_scale(0.0) == 2.0 ** -48 and oc.block_scale(3e38) == 2.0 ** 48
    for a in (1e-9, 0.3, 7.0, 1e5):
        s = oc.block_scale(a)
        assert a <= 448 * s and a > 448 * s / 2


def test_appended_values_are_within_half_a_step():
    # a value of at least 2^-6 S is off by at most 2^-4 of itself, a smaller one by at most 2^-10 S
    g = np.random.default_rng(0)
    new = (g.standard_normal((50, 2, 16)) * np.exp(g.standard_normal((50, 2, 1)))).astype(np.float32)
    codes, scales = np.zeros((4, 2, 32, 16), np.uint8), np.ones((4, 2, 2), np.float32)
    table = np.array([[2, 0, -1], [3, -1, -1]], np.int32)
    oc.append_block_scaled(codes, scales, new, table, [3, 0], [0, 40, 50], 16)
    v = oc.pool_values(codes, "e4m3", scales=scales)
    unit = np.repeat(scales, 16, axis=2)[..., None]
    for b, held, lo, n in ((0, 3, 0, 40), (1, 0, 40, 10)):
        for t in range(n):
            page, at = table[b, (held + t) // 32], (held + t) % 32
            err = np.abs(v[page, :, at] - new[lo + t])
            assert np.all(err <= np.maximum(np.abs(new[lo + t]) * 2.0 ** -4, unit[page, :, at] * 2.0 ** -10))


def test_a_growing_scale_keeps_held_values():
    # powers of two: only codes that fall under 2^-6 can change, by at most half a subnormal step
    g = np.random.default_rng(1)
    codes = g.integers(0, 0x7E, (1, 1, 16, 8), dtype=np.uint8)
    scales = np.full((1, 1, 1), 0.25, np.float32)
    before = oc.pool_values(codes, "e4m3", scales=scales)
    oc.append_block_scaled(codes, scales, np.full((1, 1, 8), 7000.0, np.float32), np.array([[0]], np.int32), [10], [0, 1], 16)
    assert scales[0, 0, 0] == 16.0
    after = oc.pool_values(codes, "e4m3", scales=scales)
    assert np.all(after[0, 0, 10] == 7168.0)                       # 7000 / 16 = 437.5, to the grid step of 32: 448
    d = np.abs(after[0, 0, :10] - before[0, 0, :10])
    assert np.all(d[before[0, 0, :10] >= 16 * 2.0 ** -6] == 0) and d.max() <= 16 * 2.0 ** -10


def test_fork_by_hand():
    # pages of 4: row 0 holds 6 positions on pages 5, 2; row 2 is overwritten and frees page 0
    table = np.array([[5, 2, -1], [-1, -1, -1], [0, -1, -1], [7, -1, -1]], np.int32)
    t, n, moves = oc.fork(table, np.array([6, 0, 3, 4]), [0, 3], [1, 2], 4, 8)
    assert moves == [(2, 0, 2)]
    assert t.tolist() == [[5, 2, -1], [5, 0, -1], [7, -1, -1], [7, -1, -1]] and n.tolist() == [6, 6, 4, 4]
    # a swap copies nothing: each reader takes the partial page of the row that is replaced
    t, n, moves = oc.fork(table, np.array([6, 0, 3, 4]), [0, 2], [2, 0], 4, 8)
    assert moves == [] and t.tolist() == [[0, -1, -1], [-1, -1, -1], [5, 2, -1], [7, -1, -1]]


def test_compact_by_hand():
    table = np.array([[6, 1, -1], [6, 3, 9]], np.int32)
    t, moves, live = oc.compact(table, [7, 5], 4, 8)
    assert live == 3 and moves == [(3, 0, 1), (6, 2, 4)]
    assert t.tolist() == [[2, 1, -1], [2, 0, 9]]


def test_attention_definition_on_two_keys():
    # weights 1 : e^1 after a cap that leaves small scores, a bias of one step, and a row that sees nothing
    k = np.zeros((1, 1, 16, 64)); v = np.zeros((1, 1, 16, 64))
    v[0, 0, 0, 0], v[0, 0, 1, 0] = 1.0, 3.0
    q = np.zeros((1, 2, 1, 64))
    out = oc.attention(q, k, v, np.array([[0]]), [2], 1.0, softcap=5.0, slopes=[1.0],
                       key_begin=np.array([[0, 0]]), key_end=np.array([[0, 2]]))
    w = np.exp(-1.0)
    assert np.all(out[0, 0] == 0) and abs(out[0, 1, 0, 0] - (w * 1 + 3) / (w + 1)) < 1e-15
    k[0, 0, 1, 0] = 10.0
    q[0, 1, 0, 0] = 100.0          # a score of 1000, capped to 5
    out = oc.attention(q, k, v, np.array([[0]]), [2], 1.0, softcap=5.0)
    w = np.exp(-5.0)
    assert abs(out[0, 1, 0, 0] - (w * 1 + 3) / (w + 1)) < 1e-12
    assert of.E4M3_MAX == 448.0


def test_a_cap_past_the_range_is_refused(lib):
    # 3e38 is finite, 3e38 log2 e is not; without the refusal scores became infinity times zero
    for f, args in ((lib.nbx_paged_decode_attn_modified, MODIFIED), (lib.nbx_paged_decode_attn_block_scaled, BLOCK)):
        assert call(f, args, softcap=3e38) == -8


def test_calls_from_an_array_of_arguments(lib):
    import struct
    assert lib.nbx_call(99, b"") == -8 and lib.nbx_call(0, None) == -1

    def packed(number, name, args, **kw):
        a = {**args, **kw}
        types = getattr(lib, name).argtypes
        raw = [getattr(v, "value", v) or 0 for v in a.values()]
        form = "=" + "".join("d" if t is ctypes.c_float else "q" for t in types)
        return lib.nbx_call(number, struct.pack(form, *raw))

    for number, (name, args) in enumerate([
            ("nbx_paged_kv_append_block_scaled", APPEND), ("nbx_paged_decode_attn_block_scaled", BLOCK),
            ("nbx_paged_decode_attn_modified", MODIFIED), ("nbx_paged_kv_copy_pages", COPY),
            ("nbx_paged_kv_fork", FORK), ("nbx_paged_kv_compact", COMPACT)]):
        for kw in (dict(num_pages=0), dict(k_pool=FAKE_ODD), dict(k_pool=NULL), dict(d=7), dict(page_tokens=0)):
            assert packed(number, name, args, **kw) == call(getattr(lib, name), args, **kw) < 0
    for kw in (dict(softcap=-1.0), dict(scale=float("nan")), dict(softcap=1e-40)):   # floats
        assert packed(2, "nbx_paged_decode_attn_modified", MODIFIED, **kw) == -8


# ------------------------------------------------------------------------- the session
def test_session_refusals():
    from paged_split_kv_append_gb300.session import PagedDecodeSession
    sizes = dict(num_pages=2, h_kv=1, page_tokens=32, d=64, batch=1, rows=1, h_q=1, max_seq_len=32, device="cpu")
    for bad in (dict(pool_dtype="bf16", scale_tokens=16), dict(pool_dtype="e4m3", scale_tokens=64),
                dict(pool_dtype="bf16", out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            PagedDecodeSession(**sizes, **bad)
    with pytest.raises(ValueError):
        PagedDecodeSession(**sizes, pool_dtype="bf16").set_modifications(softcap=1.0)
    s = PagedDecodeSession(**sizes, pool_dtype="e4m3", scale_tokens=16)
    assert s.k_scales.shape == s.v_scales.shape == (2, 1, 2) and s.modified
