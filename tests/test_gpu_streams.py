"""What a call allocates for a stream that is not the current one: memory that the current stream has freed but has
still to write to may not be handed to it, and what it fills it fills on its own stream."""

import numpy as np
import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from tests.test_gpu_modified import DEV, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    torch.cuda._sleep(1000)
    torch.zeros(1, device=DEV).fill_(7.0)      # (a kernel's first launch may wait for the device)
    torch.zeros(1, device=DEV, dtype=torch.int32).fill_(7)
    torch.cuda.synchronize()


def busy():
    torch.cuda._sleep(20_000_000)   # ten milliseconds or so of the current stream


@pytest.mark.parametrize("kind", ["plain", "modified", "block"])
def test_an_output(kind):
    c = Case("block" if kind == "block" else "bf16", "bf16", 1, 32, 8, 128, 16, (200,) * 64, 16 if kind == "block" else 0,
             seed=50)
    i32 = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    pools = [c.q.to(DEV), *c.dev] + [torch.from_numpy(x).to(DEV) for x in c.scales if x is not None]
    rest = i32(c.table), i32(c.lens), 200, c.scale
    call = {"plain": nbx.nbx_paged_decode_attn, "modified": nbx.nbx_paged_decode_attn_modified,
            "block": nbx.nbx_paged_decode_attn_block_scaled}[kind]
    ws = torch.empty(nbx.nbx_paged_decode_modified_workspace_bytes(64, 1, 32, 8, 128, 200), dtype=torch.uint8, device=DEV)
    ref = call(*pools, *rest, workspace=ws).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.empty_like(ref)
    busy()
    late.fill_(7.0)
    del late
    out = call(*pools, *rest, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_a_count_of_nothing():
    # a fork of no rows launches nothing; its zero is there when its stream is
    x = [torch.zeros((8, 1, 16, 16), device=DEV) for _ in range(2)]
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.tensor([[1, 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([20], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    spoiled = [torch.full((1,), 7, dtype=torch.int32, device=DEV) for _ in range(64)]
    torch.cuda.synchronize()
    del spoiled
    busy()
    _, count = nbx.nbx_paged_kv_fork(table, lens, none, none, *x, stream=side)
    with torch.cuda.stream(side):
        got = count.to("cpu")
    assert int(got[0]) == 0
    torch.cuda.synchronize()


def test_an_output_that_the_current_stream_still_reads():
    # the caller frees it while the current stream has still to read it; the next call on the side stream allocates
    c = Case("bf16", "bf16", 1, 32, 8, 128, 16, (200,) * 64, seed=51)
    i32 = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    args = [c.q.to(DEV), *c.dev, i32(c.table), i32(c.lens), 200, c.scale]
    other = [torch.zeros_like(args[0])] + args[1:]
    ws = torch.empty(nbx.nbx_paged_decode_modified_workspace_bytes(64, 1, 32, 8, 128, 200), dtype=torch.uint8, device=DEV)
    ref = nbx.nbx_paged_decode_attn_modified(*args, softcap=9.0, workspace=ws).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = nbx.nbx_paged_decode_attn_modified(*args, softcap=9.0, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    busy()
    copy = out.clone()
    del out
    nbx.nbx_paged_decode_attn_modified(*other, softcap=9.0, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(copy.cpu().numpy(), ref.cpu().numpy())
