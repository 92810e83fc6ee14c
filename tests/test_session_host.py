"""The session without a GPU: the scratch of its page calls, and the calls that do not fit a block-scaled cache."""

import weakref

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from paged_split_kv_append_gb300.session import PagedDecodeSession

SIZES = dict(num_pages=8, h_kv=1, page_tokens=32, d=64, batch=4, rows=1, h_q=1, max_seq_len=32, device="cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def inputs(s, width, **kw):
    s.set_inputs(torch.zeros((4, 1, 1, 64)), torch.full((4, width), -1), torch.zeros(4), None, None, None, 1.0, **kw)


def test_a_page_scratch_that_grows_keeps_the_one_before():
    # a captured graph, or a call on another stream, may still use it
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16")
    inputs(s, 4)
    first = s._page_scratch(None)
    assert s._page_scratch(None).data_ptr() == first.data_ptr()
    kept = weakref.ref(first)
    at, size = first.data_ptr(), first.numel()
    del first
    inputs(s, 4096)
    assert s._page_scratch(None).numel() > size and s._page_scratch(None).data_ptr() != at
    assert kept() is not None


def block_scaled():
    return PagedDecodeSession(**SIZES, pool_dtype="e4m3", scale_tokens=16)


def test_plain_appends_do_not_fit_a_block_scaled_cache():
    # they know nothing of the blocks' scales: the codes would stand for other values
    s = block_scaled()
    inputs(s, 4)
    x, slots = torch.zeros((2, 1, 64)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="block scales"):
        s.append(x, x, slots)
    with pytest.raises(ValueError, match="block scales"):
        s.prefill(x, x, [0, 1], [0, 1])


def test_inputs_that_do_not_fit_a_block_scaled_cache():
    s = block_scaled()
    with pytest.raises(ValueError):       # scales of a whole pool, which its decodes do not take
        inputs(s, 4, k_scale=0.5)
    with pytest.raises(ValueError):
        inputs(s, 4, v_scale=2.0)
    x = torch.zeros((2, 1, 64))
    s.set_inputs(torch.zeros((4, 1, 1, 64)), torch.full((4, 4), -1), torch.zeros(4), x, x, None, 1.0)
    with pytest.raises(ValueError, match="set_new_tokens"):       # which says where they go
        s.step()


def test_block_scaled_calls_do_not_fit_a_plain_session():
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16")
    inputs(s, 4)
    x, i = torch.zeros((2, 1, 64)), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="block scales"):
        s.append_block_scaled(x, x, i[:4], i)
    with pytest.raises(ValueError, match="block scales"):
        s.set_new_tokens(x, x, i[:4], i)
