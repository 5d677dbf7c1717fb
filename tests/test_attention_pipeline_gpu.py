"""GPU test of a sparse-attention layer's decode step as its calls are used
together: index pre-pass, key/value store, index logits, selection, attention
over the selection; one block table and slot mapping serve both caches.  Every
stage is held to the stage before it in 64 bits, and the captured step repeats
the eager one."""
import numpy as np
import pytest
import torch

from fp4_sparse_attention_fp4idx_gb300 import workloads as wl
from tests import kv_ref as R
from tests.gpu_util import F, bf16_dev, dev

pytestmark = pytest.mark.gpu


def test_decode_step():
    f = F()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rng = np.random.default_rng(5)
    B, next_n, IH, Hq, Hkv, D, k = 5, 2, 32, 16, 2, 128, 256
    ctx = [700, 64, 2, 1500, 129]  # with the step's next_n tokens
    blocks = 80
    table = R.make_table(g, ctx, blocks).clamp(min=0)
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    cos, sin = (dev(x) for x in wl.rope_tables(2048))
    cache = [torch.zeros(blocks, Hkv, 64, D, dtype=torch.uint8, device="cuda") for _ in range(2)] \
        + [torch.ones(blocks, Hkv, device="cuda") for _ in range(2)]
    index_cache = torch.zeros(blocks, 4352, dtype=torch.uint8, device="cuda")
    gamma = bf16_dev(wl.to_bf16_bits(np.ones(128)))

    def bf(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def slots_of(b, a, n):
        at = torch.arange(a, a + n, device="cuda")
        return table[b, at // 64].long() * 64 + at % 64, at

    # the prompts
    for b, c in enumerate(ctx):
        if c > next_n:
            slots, at = slots_of(b, 0, c - next_n)
            n = len(at)
            f.k_norm_rope_pack_store(bf(n, 128), gamma, at, cos, sin, slots, index_cache)
            f.kv_store_fp8(bf(n, Hkv, D), bf(n, Hkv, D), slots, *cache)
    # the step's inputs
    new = [slots_of(b, c - next_n, next_n) for b, c in enumerate(ctx)]
    slots = torch.cat([s for s, _ in new])
    pos = torch.cat([p for _, p in new])
    T = B * next_n
    ik, iq, iw = bf(T, 128), bf(T, IH, 128), bf(T, IH)
    kk, vv, q = bf(T, Hkv, D), bf(T, Hkv, D), bf(T, Hq, D)
    seen = (pos + 1).to(torch.int32)

    def step():
        f.kv_store_fp8(kk, vv, slots, *cache)
        qf, qs, wt = f.indexer_prepass(ik, gamma, slots, index_cache, iq, iw, pos, cos, sin)
        logits = f.paged_mqa_logits(qf, qs, wt, index_cache, table, lens, max(ctx), next_n=next_n)
        idx, cnt = f.topk_tokens(logits, k, row_lens=seen)
        out, lse = f.sparse_attention_fp8(q, *cache, table, idx)
        dense = f.paged_attention_fp8(q, *cache, table, lens, max(ctx))
        return logits, idx, cnt, out, lse, dense

    logits, idx, cnt, out, lse, dense = step()
    torch.cuda.synchronize()
    wi, wc = R.topk(logits, k, seen.tolist())
    assert torch.equal(idx.cpu(), wi) and torch.equal(cnt.cpu(), wc)
    assert bool((idx < seen[:, None]).all())  # no later token of the step
    seqs = [t // next_n for t in range(T)]
    ref = R.sparse(q, cache, table, idx, seqs, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, k)
    starts = [i * next_n for i in range(B + 1)]
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(dense[0].view(-1, D), dense[1].view(-1), ref, max(ctx))
    # rows whose selection is everything: both attentions saw the same keys
    whole = (cnt == seen).nonzero().squeeze(1)
    assert len(whole) > 0
    d_score = 2.0 ** -16 * ref[3].view(T, Hq) + 2.0 ** -19  # kv_ref.check's bound, twice
    lse_tol = 2 * (d_score + 2.0 ** -19 * (1 + ref[1].view(T, Hq).abs()))
    assert bool(((lse - dense[1]).double().abs() <= lse_tol)[whole].all())

    # captured: the same step, replayed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[1], idx) and torch.equal(got[3], out) and torch.equal(got[4], lse)
    assert torch.equal(got[5][0], dense[0])
