"""GPU tests of the cache operators captured together and run at once: a
decode step replayed with new inputs in place, and calls on two streams."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def step(q, k, v, slots, cache, table, lens, logits, bound):
    F().kv_store_fp8(k, v, slots, *cache)
    dense = F().paged_attention_fp8(q, *cache, table, lens, bound)
    indices, counts = F().topk_tokens(logits, 64, row_lens=lens)
    sparse = F().sparse_attention_fp8(q, *cache, table, indices)
    back = F().kv_load_fp8(*cache, slots)
    return [*dense, indices, counts, *sparse, *back]


def test_a_captured_step_replayed_with_new_inputs():
    ctx, Hq, Hkv, D = [700, 64, 3000], 16, 2, 128
    q, cache, table, _ = A.setup(ctx, [1] * 3, Hq, Hkv, D, BF, 51)
    table = table.clamp(min=0)
    lens = A.i32(ctx)
    g = A.gen(52)
    k, v = (torch.randn(3, Hkv, D, generator=g, device="cuda").to(BF) for _ in range(2))
    logits = torch.randn(3, 3000, generator=g, device="cuda")
    slots = torch.tensor([int(table[b, (c - 1) // 64]) * 64 + (c - 1) % 64
                          for b, c in enumerate(ctx)], dtype=torch.int64, device="cuda")
    start = [t.clone() for t in cache]
    args = (q, k, v, slots, cache, table, lens, logits, 3000)
    step(*args)  # sets the kernels' attributes
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*args)
    for seed in (53, 54):
        g = A.gen(seed)
        for t in (q, k, v, logits):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * 2)
        for t, s in zip(cache, start):
            t.copy_(s)
        want = [t.clone() for t in step(*args)]
        kept = [t.clone() for t in cache]
        for t, s in zip(cache, start):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, b in zip(cache, kept):
            assert torch.equal(a, b)


def test_calls_at_once_on_two_streams():
    """Prompts and single tokens over one cache, each stream's calls with
    workspaces of their own."""
    D, Hq, Hkv = 128, 32, 2
    ctx = [2000, 1500, 900, 4000]
    q, cache, table, starts = A.setup(ctx, [150] * 4, Hq, Hkv, D, BF, 61)
    lens = A.i32(ctx)
    one = q[:4].clone()
    assert 4 * 150 * Hq * (4000 // 64) > 1200 * 152  # the prompts' kernel

    def prompts():
        return F().paged_attention_fp8(q, *cache, table, lens, 4000)

    def tokens():
        return F().paged_attention_fp8(one, *cache, table, lens, 4000)

    want = prompts(), tokens()
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(want[0][0].view(-1, D), want[0][1].view(-1), ref, 4001)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(6):
        for s, call in zip(streams, (prompts, tokens)):
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(pair, want[i % 2]))
