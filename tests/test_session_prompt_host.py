"""Prompts of a session without a GPU: refused while its decodes have score modifications set."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from paged_split_kv_append_gb300.session import PagedDecodeSession

SIZES = dict(num_pages=8, h_kv=1, page_tokens=32, d=64, batch=4, rows=1, h_q=1, max_seq_len=64, device="cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()


def prompt(s):
    x = torch.zeros((4, 1, 64), dtype=torch.bfloat16)
    return s.prompt(x, x, x, torch.tensor([0, 4], dtype=torch.int32))


@pytest.mark.parametrize("made", [dict(pool_dtype="bf16", modified=True), dict(pool_dtype="e4m3", scale_tokens=16)])
@pytest.mark.parametrize("mods", [dict(softcap=30.0), dict(slopes=torch.zeros(1)), dict(key_begin=torch.zeros((4, 1), dtype=torch.int32)),
                                  dict(key_end=torch.ones((4, 1), dtype=torch.int32)), dict(softcap=0.5, slopes=torch.zeros(1))])
def test_a_prompt_beside_modified_decodes_is_refused(made, mods):
    s = PagedDecodeSession(**SIZES, **made)
    s.set_modifications(**mods)
    with pytest.raises(ValueError, match="score modification"):
        prompt(s)
    # none set any more: the call goes on to its own checks (these tensors are not on a GPU)
    s.set_modifications()
    with pytest.raises(ValueError, match="CUDA"):
        prompt(s)


def test_a_plain_session_takes_prompts():
    with pytest.raises(ValueError, match="CUDA"):
        prompt(PagedDecodeSession(**SIZES, pool_dtype="bf16"))
