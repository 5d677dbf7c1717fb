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


def test_attention_on_two_streams_without_workspaces():
    """Calls on two streams that are not the current one, each with items that
    are cut and joined through the workspace it allocates."""
    D, Hq, Hkv = 128, 16, 2
    ctx = [9000, 70, 5000]
    q, cache, table, _ = A.setup(ctx, [1] * 3, Hq, Hkv, D, BF, 71)
    table = table.clamp(min=0)
    lens = A.i32(ctx)
    other = (q.float() * -0.7).to(BF)
    idx = A.pick(A.gen(72), ctx, 3, 2048)
    calls = [
        lambda **kw: F().paged_attention_fp8(q, *cache, table, lens, 9000, **kw),
        lambda **kw: F().paged_attention_fp8(other, *cache, table, lens, 9000, **kw),
        lambda **kw: F().sparse_attention_fp8(q, *cache, table, idx, **kw),
        lambda **kw: F().sparse_attention_fp8(other, *cache, table, idx, **kw)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(40):
        for j in range(2):  # the two streams run one form with different queries
            got.append((2 * (i % 2) + j, calls[2 * (i % 2) + j](stream=streams[j])))
    torch.cuda.synchronize()
    for which, pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want[which]))


def test_workspace_is_not_taken_from_the_current_stream():
    """What the current stream allocates right behind a call on another stream
    shares no memory with the call's workspace, which may still be in use."""
    ctx, D = [9000], 128
    q, cache, table, _ = A.setup(ctx, [1], 16, 2, D, BF, 73)
    lens = A.i32(ctx)
    want = F().paged_attention_fp8(q, *cache, table, lens, 9000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = F().attention_workspace_bytes(1, 1, 16, 2, D)
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = F().paged_attention_fp8(q, *cache, table, lens, 9000, stream=side)
        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_topk_beside_a_busy_current_stream():
    """Memory that the current stream has given back but still writes does not
    become the outputs of a call on another stream."""
    x = torch.randn(64, 20000, device="cuda", generator=A.gen(5))
    want = F().topk_tokens(x, 500)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        held = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (64 * 500, 64)]
        torch.cuda._sleep(20_000_000)
        for t in held:
            t.fill_(7)
        del held, t
        got = F().topk_tokens(x, 500, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
