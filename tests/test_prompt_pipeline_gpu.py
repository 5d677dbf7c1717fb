"""GPU test of a sparse-attention layer over packed prompts as its calls are
used together: index pre-pass, key/value store, index logits of the prompts
(-inf outside each token's keys), selection without row lengths, attention over
the selection.  Every stage is held to the stage before it in 64 bits."""
import numpy as np
import pytest
import torch

from fp4_sparse_attention_fp4idx_gb300 import workloads as wl
from tests import kv_ref as R
from tests.gpu_util import F, bf16_dev, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [256, 2048])
def test_packed_prompts(k):
    f = F()
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    prompts, IH, Hq, Hkv, D = [1500, 7, 4201], 32, 16, 2, 128
    T = sum(prompts)
    begins = [sum(prompts[:i]) for i in range(len(prompts) + 1)]
    blocks = (T + 63) // 64
    pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    ks = torch.cat([torch.full((n,), b, dtype=torch.int32, device="cuda")
                    for n, b in zip(prompts, begins)])
    slots = torch.arange(T, device="cuda")  # the prompts' keys follow one another
    cos, sin = (dev(x) for x in wl.rope_tables(8192))
    cache = [torch.zeros(blocks, Hkv, 64, D, dtype=torch.uint8, device="cuda") for _ in range(2)] \
        + [torch.ones(blocks, Hkv, device="cuda") for _ in range(2)]
    index_cache = torch.zeros(blocks, 4352, dtype=torch.uint8, device="cuda")
    gamma = bf16_dev(wl.to_bf16_bits(np.ones(128)))

    def bf(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    q = bf(T, Hq, D)
    f.kv_store_fp8(bf(T, Hkv, D), bf(T, Hkv, D), slots, *cache)
    qf, qs, wt = f.indexer_prepass(bf(T, 128), gamma, slots, index_cache, bf(T, IH, 128),
                                   bf(T, IH), pos, cos, sin)
    ke = (torch.arange(T, device="cuda") + 1).to(torch.int32)
    logits = f.mqa_logits_prefill(qf, qs, wt, index_cache, ks, ke, T)
    idx, cnt = f.topk_tokens(logits, k)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    out, lse = f.sparse_attention_fp8(q, *cache, table, idx, seq_ids=torch.zeros_like(ke))
    torch.cuda.synchronize()

    assert torch.equal(cnt, (ke - ks).clamp(max=k))
    lengths = f.topk_tokens(logits, k, row_lens=ke)  # -inf before ks, nothing behind ke
    assert torch.equal(lengths[0], idx) and torch.equal(lengths[1], cnt)
    some = torch.arange(0, T, 111, device="cuda")
    wi, wc = R.topk(logits[some], k, [T] * len(some))
    assert torch.equal(idx[some].cpu(), wi) and torch.equal(cnt[some].cpu(), wc)
    ref = R.sparse(q[some], cache, table, idx[some], [0] * len(some), D ** -0.5)
    R.check(out[some].reshape(-1, D), lse[some].reshape(-1), ref, k)
