"""Waits of the attention tiles that run out: the loaders are held back for 20 ms while the other roles may wait 20 us. The
call sets the timeout bit and returns, and the next call on the same context is right. No GPU is faulted or hung: every
wait is bounded, and the delay ends by itself."""

import pytest
import torch

import paged_split_kv_append_gb300 as nbx
from test_gpu_prompt import expect, inputs, ints, near
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    nbx.build()
    yield
    nbx.nbx_set_decode_wait_test(0, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_waits_that_run_out(d):
    q, k, v = inputs(400, 4, 2, d, d)
    start, status = ints([0, 400]), ints([0])
    nbx.nbx_set_decode_wait_test(20_000, 20_000_000)
    nbx.nbx_prompt_attn(q, k, v, start, 0.1, status=status)
    torch.cuda.synchronize()
    assert int(status) & nbx.DEV_TIMEOUT
    nbx.nbx_set_decode_wait_test(0, 0)
    status.zero_()
    out = nbx.nbx_prompt_attn(q, k, v, start, 0.1, status=status)
    near(out, *expect(q, k, v, 0, 400, 0.1))
    assert int(status) == 0


@pytest.mark.parametrize("pool,out", [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_waits_that_run_out(pool, out, d):
    c = Case([(1024, [1100, 1030, 1200])], 1, 8, 2, d, 16, pool, out, d)
    status = ints([0])
    nbx.nbx_set_decode_wait_test(20_000, 20_000_000)
    c.run(status=status)
    torch.cuda.synchronize()
    assert int(status) & nbx.DEV_TIMEOUT
    nbx.nbx_set_decode_wait_test(0, 0)
    c.check_run()
