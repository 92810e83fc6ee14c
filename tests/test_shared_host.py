"""The shared-prefix decode without a GPU: what it refuses on the host before any CUDA call, and its workspace."""

import ctypes

import pytest

import paged_split_kv_append_gb300 as nbx

NULL = None
FAKE = ctypes.c_void_p(0x10000)          # a 16-byte aligned address that is never dereferenced
FAKE_ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    nbx.build()
    return nbx.lib()


CALL = dict(q=FAKE, q_dtype=1, batch=4, rows=1, h_q=8, d=128, k_pool=FAKE, v_pool=FAKE, pool_dtype=1, num_pages=100, h_kv=2,
            page_tokens=32, bt=FAKE, max_pages=10, lens=FAKE, max_seq_len=160, start=FAKE, shared=FAKE, n_groups=2, scale=0.1,
            k_scale=1.0, v_scale=1.0, out=FAKE, out_dtype=0, ws=FAKE, ws_bytes=1 << 30, status=NULL, stream=NULL)


def call(lib, **kw):
    a = dict(CALL)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.nbx_paged_decode_attn_shared(*a.values())


@pytest.mark.parametrize("want,kw", [
    (0, dict(batch=0)), (-1, dict(q=NULL)), (-1, dict(out=NULL)), (-1, dict(bt=NULL)), (-1, dict(ws=NULL)),
    (-1, dict(start=NULL)), (-1, dict(shared=NULL)), (-2, dict(n_groups=-1)), (-2, dict(h_q=9)), (-2, dict(d=96)),
    (-2, dict(rows=0)), (-2, dict(max_seq_len=321)), (-3, dict(q_dtype=2)), (-3, dict(out_dtype=2)), (-3, dict(pool_dtype=7)),
    (-4, dict(page_tokens=40, max_seq_len=100)), (-5, dict(ws_bytes=1000)), (-7, dict(out=FAKE_ODD)), (-7, dict(q=FAKE_ODD)),
    (-7, dict(ws=ctypes.c_void_p(0x10010))), (-8, dict(scale=float("nan"))), (-8, dict(scale=2e38, k_scale=100.0)),
    (-8, dict(v_scale=0.0))])
def test_refusals(lib, want, kw):
    assert call(lib, **kw) == want


def test_workspace(lib):
    f = lib.nbx_paged_decode_shared_workspace_bytes
    assert f(2, 1, 8, 3, 128, 100, 1) == 0 and f(2, 1, 8, 2, 128, 100, -1) == 0
    n = f(4, 1, 8, 2, 128, 160, 2)
    assert n >= lib.nbx_paged_decode_modified_workspace_bytes(4, 1, 8, 2, 128, 160)
    assert call(lib, ws_bytes=n - 1) == -5


def test_an_output_of_16_byte_alignment_is_refused(lib):
    assert call(lib, out=ctypes.c_void_p(0x10010)) == -7
    assert call(lib, out=ctypes.c_void_p(0x10010), n_groups=0) == -7
