"""GPU tests of calls on a stream that is not the current one: what a call
allocates is in order with its own stream, whatever the current one does."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_load_beside_a_busy_current_stream():
    g = A.gen(3)
    cache = R.make_cache(g, 9, 2, 128)
    slots = torch.randperm(9 * 64, generator=g, device="cuda")[:300]
    slots[::7] = -1
    want = F().kv_load_fp8(*cache, slots)
    assert bool((want[0][::7] == 0).all()) and bool((want[0] != 0).any())
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        got = F().kv_load_fp8(*cache, slots, stream=side)
        side.synchronize()
        early = [t.clone() for t in got]  # behind the sleep
        torch.cuda.synchronize()
        for a, b, c in zip(got, early, want):
            assert torch.equal(a, c) and torch.equal(b, c)
