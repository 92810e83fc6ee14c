"""Prompt attention without a GPU: what it refuses on the host before any CUDA call."""

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


CALL = dict(q=FAKE, q_stride=1024, k=FAKE, k_stride=256, v=FAKE, v_stride=256, dtype=1, n_tok=40, h_q=8, h_kv=2, d=128,
            start=FAKE, batch=3, scale=0.1, out=FAKE, status=NULL, stream=NULL)


@pytest.mark.parametrize("want,kw", [
    (0, dict(n_tok=0)), (0, dict(batch=0)), (-1, dict(q=NULL)), (-1, dict(k=NULL)), (-1, dict(v=NULL)),
    (-1, dict(start=NULL)), (-1, dict(out=NULL)), (-2, dict(n_tok=-1)), (-2, dict(batch=-1)), (-2, dict(h_q=0)),
    (-2, dict(h_kv=0)), (-2, dict(h_kv=3)), (-2, dict(d=96)), (-2, dict(d=32)), (-2, dict(q_stride=1000)),
    (-2, dict(k_stride=252)), (-2, dict(v_stride=260)), (-3, dict(dtype=0)), (-3, dict(dtype=2)), (-7, dict(q=FAKE_ODD)),
    (-7, dict(v=FAKE_ODD)), (-7, dict(out=FAKE_ODD)), (-7, dict(out=ctypes.c_void_p(0x10010))), (-8, dict(scale=float("nan"))), (-8, dict(scale=float("inf"))),
    (-8, dict(scale=3e38))])
def test_refusals(lib, want, kw):
    a = dict(CALL)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.nbx_prompt_attn(*a.values()) == want


def test_the_binding_refuses_host_tensors():
    x = torch.zeros((4, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nbx.nbx_prompt_attn(x, x, x, torch.zeros(2, dtype=torch.int32), 1.0)


def far(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.mark.parametrize("kw", [
    dict(out=FAKE), dict(out=far(40 * 2048 - 32)), dict(q=far(1 << 20), out=far(39 * 512 + 480)),
    dict(q=far(1 << 20), k=far(1 << 21), out=far(32)), dict(q=far(40 * 2048 - 16), k=far(1 << 21), v=far(1 << 22)),
    dict(n_tok=1, q_stride=0, k_stride=0, v_stride=0, out=far(2016))], ids=str)
def test_an_output_over_an_input_is_refused(lib, kw):
    a = dict(CALL)
    a.update(kw)
    assert lib.nbx_prompt_attn(*a.values()) == -8
