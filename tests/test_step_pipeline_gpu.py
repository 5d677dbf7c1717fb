"""GPU test of serving steps as their calls are used together: pages and maps, rotary
positions, the store, attention of whole prompts, then padded decode steps (captured
and replayed) with selection, attention over the cache and over the selection, and
pages given back.  Every stage is held to the stage before it in 64 bits."""
import pytest
import torch

from tests import kv_ref as K
from tests import step_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
B, H, HK, D, WIDTH, BLOCKS = 5, 8, 2, 128, 12, 40
SECTIONS = (24, 20, 20)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self):
        g = self.g = torch.Generator(device="cuda")
        g.manual_seed(3)
        self.cache = [torch.zeros(BLOCKS, HK, 64, D, dtype=torch.uint8, device="cuda")
                      for _ in range(2)] + [torch.ones(BLOCKS, HK, device="cuda") for _ in range(2)]
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(BLOCKS, generator=g, device="cuda").to(torch.int32)
        self.count = i32([BLOCKS])
        self.lens = i32([0] * B)
        inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
        a = torch.arange(2048, dtype=torch.float64, device="cuda")[:, None] * inv
        self.cos, self.sin = a.cos().float(), a.sin().float()
        self.err = i32([0])

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(BF)

    def extend(self, new, T):
        return F().batch_extend(self.lens, new, self.table, self.free, self.count, T,
                                err_flags=self.err)

    def store(self, qkv, maps):
        """The projection's rows turned and stored; queries, keys, values."""
        axes = torch.stack([maps.positions, maps.positions // 7, maps.positions % 7])
        q, k, v = qkv[:, :H], qkv[:, H:H + HK], qkv[:, H + HK:]
        q, k = F().rope_qk(q, k, axes, self.cos, self.sin, sections=SECTIONS, err_flags=self.err)
        F().kv_store_fp8(k, v, maps.slot_mapping, *self.cache, err_flags=self.err)
        return q, k, v


def test_prompts_then_decode_steps():
    f, s = F(), Layer()
    prompts = [130, 0, 64, 300, 1]
    qs = [sum(prompts[:i]) for i in range(B + 1)]
    T = sum(prompts) + 9
    qkv = s.rand(T, H + 2 * HK, D)

    # ---- the prompts, padded by nine rows of garbage
    qkv[-9:] = float("nan")
    maps = s.extend(i32(prompts), T)
    q, k, v = s.store(qkv, maps)
    out = torch.full((T, H, D), 5.0, dtype=BF, device="cuda")
    out, lse = f.prompt_attention(q, k, v, maps.q_starts, max(prompts), out=out, err_flags=s.err)
    assert maps.q_starts.tolist() == qs and int(s.err) == 0
    n = qs[-1]
    pos = torch.cat([torch.arange(p, device="cuda") for p in prompts])
    axes = torch.stack([pos, pos // 7, pos % 7])
    for got, x in ((q, qkv[:, :H]), (k, qkv[:, H:H + HK])):
        want, _ = R.rope(x[:n], axes, s.cos, s.sin, list(SECTIONS), False, True, torch.float32)
        assert torch.equal(got[:n], want.to(BF))
    R.check(out[:n], lse[:n], R.attend(q[:n], k[:n], v[:n], qs, qs, 0, 0, D ** -0.5))
    assert bool((out[n:] == 5).all())
    s.lens.copy_(maps.context_lens)
    assert s.lens.tolist() == prompts

    # ---- decode steps of two tokens each but for one sequence that pauses; the
    # step is padded to 12 tokens and captured
    new = i32([2, 2, 2, 0, 2])
    TD = 12
    x, logits = s.rand(TD, H + 2 * HK, D), torch.randn(TD, 700, device="cuda")

    def step():
        maps = s.extend(new, TD)
        q, k, v = s.store(x, maps)
        idx, cnt = f.topk_tokens(logits, 50, row_lens=maps.row_lens)
        dense = f.paged_attention_fp8(q, *s.cache, s.table, maps.context_lens, 700,
                                      q_starts=maps.q_starts, max_q=2, err_flags=s.err)
        sparse = f.sparse_attention_fp8(q, *s.cache, s.table, idx, seq_ids=maps.seq_ids,
                                        err_flags=s.err)
        s.lens.copy_(maps.context_lens)
        return maps, q, idx, cnt, dense, sparse

    state = [t.clone() for t in (*s.cache, s.table, s.count, s.lens)]
    step()  # loads the kernels
    torch.cuda.synchronize()
    for t, was in zip((*s.cache, s.table, s.count, s.lens), state):
        t.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        maps, q, idx, cnt, dense, sparse = step()
    lens = list(prompts)
    for _ in range(40):
        x.copy_(s.rand(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert int(s.err) == 0
        lens = [c + a for c, a in zip(lens, new.tolist())]
        assert s.lens.tolist() == lens
        starts = [0, 2, 4, 6, 6, 8]
        assert maps.q_starts.tolist() == starts
        want = [(b, lens[b] - 2 + i) for b in (0, 1, 2, 4) for i in range(2)]
        assert maps.seq_ids.tolist() == [b for b, _ in want] + [0] * 4
        assert maps.positions.tolist() == [p for _, p in want] + [0] * 4
        assert maps.row_lens.tolist() == [p + 1 for _, p in want] + [0] * 4
        assert maps.slot_mapping.tolist() == \
            [int(s.table[b, p // 64]) * 64 + p % 64 for b, p in want] + [-1] * 4
    held = sum(R.pages(c) for c in lens)
    assert int(s.count) == BLOCKS - held
    used = s.table[s.table >= 0].tolist()
    assert len(used) == len(set(used)) == held
    wi, wc = K.topk(logits, 50, maps.row_lens.tolist())
    assert torch.equal(idx.cpu(), wi) and torch.equal(cnt.cpu(), wc)
    ref = K.dense(q[:8], s.cache, s.table, lens, starts, 0, 0, D ** -0.5)
    K.check(dense[0][:8].view(-1, D), dense[1][:8].view(-1), ref, max(lens))
    ref = K.sparse(q[:8], s.cache, s.table, idx[:8], maps.seq_ids.tolist()[:8], D ** -0.5)
    K.check(sparse[0][:8].view(-1, D), sparse[1][:8].view(-1), ref, 50)

    # ---- the same tokens' prompt attention over the cache's own values: the cache
    # read back in 16 bits is the contiguous keys of a chunk
    slots = torch.cat([s.table[b, torch.arange(c, device="cuda") // 64].long() * 64 +
                       torch.arange(c, device="cuda") % 64 for b, c in enumerate(lens)])
    k16, v16 = f.kv_load_fp8(*s.cache, slots)
    ks = [sum(lens[:i]) for i in range(B + 1)]
    out, lse = f.prompt_attention(q, k16, v16, maps.q_starts, 2, k_starts=i32(ks), max_k=max(lens))
    ref = R.attend(q[:8], k16, v16, starts, ks, 0, 0, D ** -0.5)
    R.check(out[:8], lse[:8], ref)

    # ---- two sequences end, one gives back rejected drafts
    kept = [0, lens[1], lens[2] - 65, lens[3], 0]
    f.pages_release(s.lens, i32(kept), s.table, s.free, s.count, err_flags=s.err)
    assert int(s.err) == 0 and int(s.count) == BLOCKS - sum(R.pages(c) for c in kept)
    free = s.free[:int(s.count)].tolist()
    used = s.table[s.table >= 0].tolist()
    assert sorted(free + used) == list(range(BLOCKS))
