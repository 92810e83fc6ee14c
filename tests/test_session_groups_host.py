"""Sessions whose decodes share prefixes, without a GPU: what they are made with, and what does not go with it."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from paged_split_kv_append_gb300.session import PagedDecodeSession

SIZES = dict(num_pages=8, h_kv=1, page_tokens=32, d=64, batch=4, rows=1, h_q=1, max_seq_len=64, device="cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def test_the_workspace_holds_the_groups():
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16", shared_groups=2)
    assert s.workspace.numel() >= nbx.nbx_paged_decode_shared_workspace_bytes(4, 1, 1, 1, 64, 64, 2)
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16", shared_groups=2, out_dtype=torch.bfloat16)
    assert s.out.dtype is torch.bfloat16


def test_what_does_not_go_together():
    with pytest.raises(ValueError, match="plain"):
        PagedDecodeSession(**SIZES, pool_dtype="bf16", shared_groups=2, modified=True)
    with pytest.raises(ValueError, match="plain"):
        PagedDecodeSession(**SIZES, pool_dtype="e4m3", shared_groups=2, scale_tokens=16)
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16")
    with pytest.raises(ValueError, match="groups"):
        s.set_groups(ints([0, 4]), ints([32]))
    s.set_groups(None, None)
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16", shared_groups=1)
    with pytest.raises(ValueError, match="groups"):
        s.set_groups(ints([0, 2, 4]), ints([32, 32]))
    s = PagedDecodeSession(**SIZES, pool_dtype="e4m3", scale_tokens=16)
    x = torch.zeros((1, 1, 64))
    with pytest.raises(ValueError, match="append_rotated"):
        s.append_rotated(None, x, x, torch.zeros(4, 32), torch.zeros(4, 32), ints([0]), ints([0]))
