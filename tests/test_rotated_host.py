"""The rotated append without a GPU: what it refuses on the host before any CUDA call."""

import ctypes

import pytest
import torch

import paged_split_kv_append_gb300 as nbx

NULL = None
FAKE = ctypes.c_void_p(0x10000)          # a 16-byte aligned address that is never dereferenced
FAKE_ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    nbx.build()
    return nbx.lib()


CALL = dict(q=FAKE, q_stride=1024, h_q=8, new_k=FAKE, k_stride=256, new_v=FAKE, v_stride=256, new_dtype=1, n_tok=4, h_kv=2,
            d=128, cos=FAKE, sin=FAKE, n_pos=100, turned=128, interleaved=0, positions=FAKE, q_out=FAKE, q_out_stride=1024,
            k_out=FAKE, k_out_stride=256, k_pool=FAKE, v_pool=FAKE, pool_dtype=1, num_pages=8, page_tokens=16, slots=FAKE, k_scale=1.0, v_scale=1.0,
            status=NULL, stream=NULL)


@pytest.mark.parametrize("want,kw", [
    (0, dict(n_tok=0)), (-1, dict(q=NULL)), (-1, dict(q_out=NULL)), (-1, dict(new_k=NULL)), (-1, dict(new_v=NULL)),
    (-1, dict(cos=NULL)), (-1, dict(sin=NULL)), (-1, dict(positions=NULL)), (-1, dict(k_pool=NULL)),
    (-1, dict(v_pool=NULL)), (-1, dict(slots=NULL)), (-2, dict(n_tok=-1)), (-2, dict(h_q=-1)), (-2, dict(h_kv=0)),
    (-2, dict(d=8)), (-2, dict(d=72)), (-2, dict(d=2048)), (-2, dict(num_pages=0)), (-2, dict(page_tokens=0)),
    (-2, dict(n_pos=0)), (-2, dict(turned=0)), (-2, dict(turned=24)), (-2, dict(turned=144)), (-2, dict(q_stride=1016)),
    (-2, dict(k_stride=255)), (-2, dict(v_stride=260)), (-2, dict(q_out_stride=1028)), (-3, dict(new_dtype=2)),
    (-3, dict(pool_dtype=5)), (-2, dict(k_out_stride=252)), (0, dict(k_out_stride=252, n_tok=0, k_out=NULL)), (-7, dict(q=FAKE_ODD)), (-7, dict(k_out=FAKE_ODD)), (-7, dict(sin=FAKE_ODD)), (-7, dict(k_pool=FAKE_ODD)),
    (-8, dict(k_scale=0.0)), (-8, dict(v_scale=float("inf"))), (-8, dict(interleaved=2))])
def test_refusals(lib, want, kw):
    a = dict(CALL)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.nbx_paged_kv_append_rotated(*a.values()) == want


def test_the_binding_refuses_host_tensors():
    x = torch.zeros((1, 1, 64))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nbx.nbx_paged_kv_append_rotated(None, x, x, torch.zeros(4, 32), torch.zeros(4, 32), i, torch.zeros(1, 1, 16, 64),
                                        torch.zeros(1, 1, 16, 64), i)


@pytest.mark.parametrize("kw", [dict(q_out_stride=2048), dict(q_stride=2048), dict(k_out_stride=512),
                                dict(k_stride=512, k_out_stride=256)], ids=str)
def test_in_place_with_another_stride_is_refused(lib, kw):
    a = dict(CALL)
    a.update(kw)
    assert lib.nbx_paged_kv_append_rotated(*a.values()) == -8
