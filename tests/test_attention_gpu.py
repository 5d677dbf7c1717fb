"""GPU tests of attention over the 8-bit cache, dense and over selected
tokens, against the 64-bit definition within derived bounds (kv_ref.check)."""
import pytest
import torch

from tests import kv_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
ERR_PAGE = 0x8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def setup(ctx, qs, Hq, Hkv, D, dtype, seed, spread=0.5):
    g = gen(seed)
    blocks = sum((c + 63) // 64 for c in ctx) + 2
    cache = R.make_cache(g, blocks, Hkv, D, spread)
    table = R.make_table(g, ctx, blocks)
    starts = [sum(qs[:i]) for i in range(len(qs) + 1)]
    q = (torch.randn(starts[-1], Hq, D, generator=g, device="cuda") * 1.5).to(dtype)
    # bytes behind a context are garbage, NaN codes among them
    kc, vc, ks, vs = cache
    for b, c in enumerate(ctx):
        if c % 64:
            page = int(table[b, c // 64])
            kc[page, :, c % 64:] = R.NAN_CODE
            vc[page, :, c % 64:] = 0xFF
    return q, cache, table, starts


def run_dense(ctx, qs, Hq, Hkv, D, dtype, window=0, sinks=0, seed=0, spread=0.5, scale=None,
              ragged=True):
    q, cache, table, starts = setup(ctx, qs, Hq, Hkv, D, dtype, seed, spread)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(q_starts=i32(starts), max_q=max(qs)) if ragged else {}
    out, lse = F().paged_attention_fp8(q, *cache, table, i32(ctx), max(max(ctx), 1), window=window,
                                       sinks=sinks, softmax_scale=scale, err_flags=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref = R.dense(q, cache, table, ctx, starts, window, sinks, scale or D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, max(ctx) + 1)
    return out, lse


@pytest.mark.parametrize("ctx", [[1], [63], [64], [65], [0], [129, 0, 7], [1000, 1, 513]])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 1, 128, BF), (6, 2, 64, HF), (12, 12, 128, HF),
                                            (14, 2, 128, BF), (32, 2, 64, BF), (48, 2, 128, BF),
                                            (40, 1, 64, HF)])
def test_decode(ctx, Hq, Hkv, D, dtype):
    run_dense(ctx, [1] * len(ctx), Hq, Hkv, D, dtype, ragged=False, seed=sum(ctx) + Hq)


@pytest.mark.parametrize("n", [2, 4, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (64, 4), (100, 70), (129, 0), (5000, 3)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, BF), (7, 1, 64, HF)])
def test_drafted_tokens(n, window, sinks, Hq, Hkv, D, dtype):
    """Several query tokens a sequence, causal, with windows; contexts shorter
    than the query leave rows without a key."""
    ctx = [700, n, n - 1, 1, 0, 64 + n, 257]
    run_dense(ctx, [n] * len(ctx), Hq, Hkv, D, dtype, window, sinks, ragged=False, seed=n + window)


@pytest.mark.parametrize("window,sinks", [(0, 0), (77, 5)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 1, 128, BF), (6, 2, 64, HF), (16, 2, 128, HF)])
def test_ragged_prefill(window, sinks, Hq, Hkv, D, dtype):
    qs = [130, 0, 1, 257, 64, 3]
    ctx = [130, 55, 1, 700, 100, 640]
    run_dense(ctx, qs, Hq, Hkv, D, dtype, window, sinks, seed=window + Hq)


@pytest.mark.parametrize("ctx,qs", [([128], [128]), ([129], [129]), ([1], [1]), ([300], [40]),
                                    ([1000, 77], [64, 77]), ([513, 0, 640], [513, 0, 5]),
                                    ([2000], [33])])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,window,sinks", [
    (8, 2, 128, BF, 0, 0), (3, 1, 64, HF, 0, 0), (5, 1, 128, HF, 130, 0), (8, 1, 64, BF, 50, 200),
    (130, 1, 128, BF, 0, 0), (260, 2, 64, BF, 300, 4), (1, 1, 128, BF, 1, 1)])
def test_prompts(ctx, qs, Hq, Hkv, D, dtype, window, sinks):
    """Chunks and whole prompts, up to 1,200 rows a key head: the tensor-core
    kernel's row halves, tile borders, masks and key ranges."""
    run_dense(ctx, qs, Hq, Hkv, D, dtype, window, sinks, seed=Hq + window + sum(ctx))


def test_prompt_longer_than_the_context_it_is_given():
    """A context shorter than the chunk leaves the first rows without a key."""
    run_dense([100, 40, 0], [160, 160, 160], 4, 1, 128, BF, ragged=False, seed=2)


def test_tokens_behind_max_q_are_left_unwritten():
    ctx, D = [400], 64
    q, cache, table, starts = setup(ctx, [200], 4, 2, D, BF, 31)
    for max_q in (7, 100):
        out = torch.full((200, 4, D), 3.0, dtype=BF, device="cuda")
        lse = torch.full((200, 4), 3.0, device="cuda")
        F().paged_attention_fp8(q, *cache, table, i32(ctx), 400, q_starts=i32(starts), max_q=max_q,
                                out=out, lse=lse)
        ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
        ref = tuple(x.view(200, 4, -1)[:max_q].reshape(-1, *x.shape[1:]) for x in ref)
        R.check(out[:max_q].reshape(-1, D), lse[:max_q].reshape(-1), ref, 401)
        assert bool((out[max_q:] == 3.0).all()) and bool((lse[max_q:] == 3.0).all())


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_bad_pages_in_a_prompt(bad):
    ctx, D, n = [500], 128, 50
    q, cache, table, starts = setup(ctx, [n], 8, 2, D, BF, 32)
    t = table.clone()
    t[0, 3] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = F().paged_attention_fp8(q, *cache, t, i32(ctx), 500, err_flags=err)
    assert int(err.item()) == ERR_PAGE
    idx = torch.full((n, 500), -1, dtype=torch.int32)
    for i in range(n):
        keep = [s for s in range(500 - n + i + 1) if s // 64 != 3]
        idx[i, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
    ref = R.sparse(q, cache, table, idx.cuda(), [0] * n, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, 501)


@pytest.mark.parametrize("mag,scale", [(30.0, None), (1e-3, -0.5), (1.0, 0.0)])
def test_prompt_magnitudes_and_scales(mag, scale):
    ctx, D = [333, 260], 128
    q, cache, table, starts = setup(ctx, [64, 64], 8, 2, D, BF, 5)
    q = (q.float() * mag).to(BF)
    out, lse = F().paged_attention_fp8(q, *cache, table, i32(ctx), 333, softmax_scale=scale)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5 if scale is None else scale)
    R.check(out.view(-1, D), lse.view(-1), ref, 334)


def test_prompt_deterministic_and_captured():
    ctx, D = [3000], 128
    q, cache, table, starts = setup(ctx, [100], 8, 2, D, BF, 41)
    first = F().paged_attention_fp8(q, *cache, table, i32(ctx), 3000)
    graph = torch.cuda.CUDAGraph()
    lens = i32(ctx)
    with torch.cuda.graph(graph):
        got = F().paged_attention_fp8(q, *cache, table, lens, 3000)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("Hq,Hkv,D,dtype,n", [(8, 1, 128, BF, 1), (16, 2, 64, HF, 1),
                                              (4, 4, 128, BF, 3), (32, 1, 128, BF, 1)])
def test_long_contexts_are_split_and_joined(Hq, Hkv, D, dtype, n):
    run_dense([20011, 3, 8192, 0], [n] * 4, Hq, Hkv, D, dtype, ragged=False, seed=Hq)


def test_more_sequences_than_threads():
    ctx = [(i * 37) % 150 for i in range(700)]
    run_dense(ctx, [1] * 700, 2, 1, 64, BF, ragged=False, seed=1)


@pytest.mark.parametrize("n", [1, 40])
def test_page_scales_far_apart(n):
    """Pages whose scales lie 2^80 apart, and pages of zeros (scale 2^-126)."""
    ctx, Hq, Hkv, D = [640, 300], 8, 2, 128
    q, cache, table, starts = setup(ctx, [n, n], Hq, Hkv, D, BF, 3)
    kc, vc, ks, vs = cache
    for b, c in enumerate(ctx):
        for p in range((c + 63) // 64):
            page = int(table[b, p])
            if p % 3 == 1:
                vs[page] *= 2.0 ** (40 if b else -40)
            if p % 3 == 2:
                vc[page] = 0
                vs[page] = 2.0 ** -126
    out, lse = F().paged_attention_fp8(q, *cache, table, i32(ctx), 640)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, 641)


@pytest.mark.parametrize("mag", [1e-30, 1e-3, 30.0])
def test_query_magnitudes_and_scales(mag):
    """Tiny queries (uniform attention) and large ones (one key takes all)."""
    ctx, D = [333, 65], 128
    q, cache, table, starts = setup(ctx, [1, 1], 8, 2, D, BF, 5)
    q = (q.float() * mag).to(BF)
    for scale in (D ** -0.5, -0.3, 0.0):
        out, lse = F().paged_attention_fp8(q, *cache, table, i32(ctx), 333, softmax_scale=scale)
        ref = R.dense(q, cache, table, ctx, starts, 0, 0, scale)
        R.check(out.view(-1, D), lse.view(-1), ref, 334)


def test_one_key_takes_the_weight_of_a_long_tail():
    """A first token that holds most of the weight against a long flat tail:
    the tail's mass must not vanish by rounding."""
    ctx, D = [30000], 128
    q, cache, table, starts = setup(ctx, [1], 8, 1, D, BF, 6, spread=0.0)
    kc, vc, ks, vs = cache
    q[:] = 0
    q[..., 0] = 12.0
    kc[int(table[0, 0]), :, 0] = 0
    kc[int(table[0, 0]), :, 0, 0] = 0x7E  # 448
    out, lse = F().paged_attention_fp8(q, *cache, table, i32(ctx), 30000)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, 30001)


def test_bad_pages_are_left_out_and_flagged():
    ctx, D = [300], 64
    q, cache, table, starts = setup(ctx, [1], 4, 2, D, BF, 8)
    good = F().paged_attention_fp8(q, *cache, table, i32([300]), 300)
    for bad in (-1, cache[0].shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = F().paged_attention_fp8(q, *cache, t, i32([300]), 300, err_flags=err)
        assert int(err.item()) == ERR_PAGE
        keep = [i for i in range(300) if i // 64 != 2]
        ref = R.sparse(q, cache, table, i32([keep]), [0], D ** -0.5)
        R.check(out.view(-1, D), lse.view(-1), ref, 301)
    assert bool(torch.isfinite(good[0].float()).all())


def test_strided_queries_and_given_outputs():
    """q as a view of a packed projection; outputs and workspace given; rows
    behind the last sequence left as they were."""
    ctx, D, Hq, Hkv = [100, 200], 128, 4, 1
    q, cache, table, starts = setup(ctx, [3, 2], Hq, Hkv, D, BF, 9)
    packed = torch.randn(7, Hq + 3, D, device="cuda").to(BF)
    packed[:5, 1:1 + Hq] = q
    qv = packed[:, 1:1 + Hq]
    out = torch.full((7, Hq, D), 5.0, dtype=BF, device="cuda")
    lse = torch.full((7, Hq), 5.0, device="cuda")
    ws = torch.empty(F().attention_workspace_bytes(2, 3, Hq, Hkv, D), dtype=torch.uint8,
                     device="cuda")
    F().paged_attention_fp8(qv, *cache, table, i32(ctx), 200, q_starts=i32(starts), max_q=3,
                            out=out, lse=lse, workspace=ws)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(out[:5].view(-1, D), lse[:5].view(-1), ref, 201)
    assert bool((out[5:] == 5.0).all()) and bool((lse[5:] == 5.0).all())


def pick(g, ctx, T, k, holes=True):
    rows = []
    for t in range(T):
        n = ctx[t]
        at = torch.randperm(n, generator=g, device="cuda")[:k].to(torch.int32)
        row = torch.full((k,), -1, dtype=torch.int32, device="cuda")
        row[:len(at)] = at
        if holes:
            row = row[torch.randperm(k, generator=g, device="cuda")]
            row[::11] = -1
        rows.append(row)
    return torch.stack(rows).contiguous() if k else torch.empty(T, 0, dtype=torch.int32,
                                                                device="cuda")


@pytest.mark.parametrize("k", [1, 31, 64, 100, 700, 2048])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 1, 128, BF), (6, 2, 64, HF), (32, 2, 128, HF),
                                            (64, 2, 128, BF), (5, 5, 64, BF), (40, 1, 64, HF)])
def test_selected_tokens(k, Hq, Hkv, D, dtype):
    ctx = [900, 5, 64, 1, 3000]
    q, cache, table, _ = setup(ctx, [1] * 5, Hq, Hkv, D, dtype, k)
    table = table.clamp(min=0)
    idx = pick(gen(k), ctx, 5, k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = F().sparse_attention_fp8(q, *cache, table, idx, err_flags=err)
    ref = R.sparse(q, cache, table, idx, [0, 1, 2, 3, 4], D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, k + 1)
    assert int(err.item()) == 0


def test_selected_tokens_of_named_sequences_and_repeated_entries():
    ctx, D = [500, 300], 128
    q, cache, table, _ = setup(ctx, [9, 8], 16, 2, D, BF, 3)
    seqs = [1, 0, 0, 1, 1, 0, 1, 0, 0, 0, 1, 1, 0, 1, 0, 1, 0]
    idx = torch.randint(0, 300, (17, 150), device="cuda", dtype=torch.int32)
    idx[:, 50:60] = idx[:, :10]  # twice
    idx[3] = -1  # nothing selected
    out, lse = F().sparse_attention_fp8(q, *cache, table.clamp(min=0), idx, seq_ids=i32(seqs))
    ref = R.sparse(q, cache, table.clamp(min=0), idx, seqs, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, 151)
    # consecutive tokens per sequence by default
    one = F().sparse_attention_fp8(q[:16], *cache, table.clamp(min=0), idx[:16])
    two = F().sparse_attention_fp8(q[:16], *cache, table.clamp(min=0), idx[:16],
                                   seq_ids=i32([0] * 8 + [1] * 8))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_selection_out_of_range_is_left_out_and_flagged():
    ctx, D = [200, 200], 64
    q, cache, table, _ = setup(ctx, [1, 1], 4, 1, D, BF, 4)
    idx = torch.arange(200, device="cuda", dtype=torch.int32).repeat(2, 1)
    for change, seqs in ((64 * table.shape[1], [0, 1]), (2 ** 31 - 1, [0, 1]), (None, [0, 2]),
                         (None, [-1, 1])):
        bad = idx.clone()
        if change is not None:
            bad[0, 77] = change
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = F().sparse_attention_fp8(q, *cache, table, bad, seq_ids=i32(seqs),
                                            err_flags=err)
        assert int(err.item()) == ERR_PAGE
        want = idx.clone()
        if change is not None:
            want[0, 77] = -1
        for t, s in enumerate(seqs):
            if not 0 <= s < 2:
                want[t] = -1
        ref = R.sparse(q, cache, table, want, [0, 1], D ** -0.5)
        R.check(out.view(-1, D), lse.view(-1), ref, 201)


def test_no_selection_at_all():
    q, cache, table, _ = setup([100], [1], 4, 1, 64, BF, 4)
    out, lse = F().sparse_attention_fp8(q, *cache, table, torch.empty(1, 0, dtype=torch.int32,
                                                                      device="cuda"))
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_selecting_every_token_is_dense_attention():
    """Both forms over the same keys agree within both bounds."""
    ctx, D = [777], 128
    q, cache, table, starts = setup(ctx, [1], 8, 2, D, BF, 14)
    idx = torch.arange(777, device="cuda", dtype=torch.int32)[None]
    a = F().sparse_attention_fp8(q, *cache, table, idx)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(a[0].view(-1, D), a[1].view(-1), ref, 778)


def test_runs_are_deterministic_and_streams_are_respected():
    ctx, D = [9000, 100, 4000], 128
    q, cache, table, starts = setup(ctx, [1] * 3, 16, 2, D, BF, 21)
    args = (*cache, table, i32(ctx), 9000)
    first = F().paged_attention_fp8(q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = F().paged_attention_fp8(q, *args)
    third = F().paged_attention_fp8(q, *args, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for other in (second, third):
        assert torch.equal(first[0], other[0]) and torch.equal(first[1], other[1])


def test_captured_and_replayed():
    """Two graphs, each with a workspace of its own, replayed on two streams
    with new inputs in place."""
    ctx, D = [5000, 64], 128
    q, cache, table, starts = setup(ctx, [1] * 2, 16, 2, D, BF, 22)
    lens = i32(ctx)
    idx = pick(gen(1), ctx, 2, 300)
    F().paged_attention_fp8(q, *cache, table, lens, 5000)
    F().sparse_attention_fp8(q, *cache, table.clamp(min=0), idx)
    graphs = []
    tab = table.clamp(min=0)
    for form in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if form == 0:
                got = F().paged_attention_fp8(q, *cache, table, lens, 5000)
            else:
                got = F().sparse_attention_fp8(q, *cache, tab, idx)
        graphs.append((graph, got))
    q.copy_(torch.randn_like(q.float()).to(BF))
    lens.copy_(i32([4100, 3]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, (graph, _) in zip(streams, graphs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    ref = R.dense(q, cache, table, [4100, 3], starts, 0, 0, D ** -0.5)
    R.check(graphs[0][1][0].view(-1, D), graphs[0][1][1].view(-1), ref, 5001)
    ref = R.sparse(q, cache, tab, idx, [0, 1], D ** -0.5)
    R.check(graphs[1][1][0].view(-1, D), graphs[1][1][1].view(-1), ref, 301)


def test_empty_calls():
    q, cache, table, _ = setup([10], [1], 4, 1, 64, BF, 4)
    out, lse = F().paged_attention_fp8(q[:0], *cache, table[:0], i32([]), 64)
    assert out.shape == (0, 4, 64)
    out, lse = F().sparse_attention_fp8(q[:0], *cache, table[:0],
                                        torch.empty(0, 5, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)
