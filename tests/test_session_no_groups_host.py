"""Decodes of a session made for groups while none is set, without a GPU: what the call is given."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from paged_split_kv_append_gb300 import session
from paged_split_kv_append_gb300.session import PagedDecodeSession

SIZES = dict(num_pages=8, h_kv=1, page_tokens=32, d=64, batch=4, rows=1, h_q=1, max_seq_len=64, device="cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def test_a_decode_without_groups_makes_no_tensor(monkeypatch):
    """The empty groups are made with the session, not in each decode, whose stream would not be theirs."""
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16", shared_groups=2)
    given = []

    def fake(q, k_pool, v_pool, table, lens, max_len, start, shared, *args, **kw):
        given.append((start, shared))
        return kw["out"]

    def no_more(*args, **kw):
        raise AssertionError("a decode made a tensor")

    monkeypatch.setattr(session, "nbx_paged_decode_attn_shared", fake)
    for name in ("zeros", "empty", "full", "tensor", "as_tensor"):
        monkeypatch.setattr(session.torch, name, no_more)
    assert s.decode() is s.out and s.decode() is s.out
    monkeypatch.undo()
    (start, shared), again = given[0], given[1]
    assert start is again[0] and shared is again[1]
    assert start.dtype is shared.dtype is torch.int32 and start.tolist() == [0] and shared.numel() == 0
    groups = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([32], dtype=torch.int32)
    monkeypatch.setattr(session, "nbx_paged_decode_attn_shared", fake)
    s.set_groups(*groups)
    s.decode()
    assert given[2][0] is groups[0] and given[2][1] is groups[1]
    s.set_groups(None, None)
    s.decode()
    assert given[3][0] is start and given[3][1] is shared


def test_half_of_the_groups_is_refused():
    s = PagedDecodeSession(**SIZES, pool_dtype="bf16", shared_groups=2)
    x = torch.tensor([0, 4], dtype=torch.int32)
    for half in ((x, None), (None, x[:1])):
        with pytest.raises(ValueError, match="both or neither"):
            s.set_groups(*half)
        assert s.groups is None
