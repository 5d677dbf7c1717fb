"""GPU tests of the kernel that takes dense attention of much work: the cases
that few rows take elsewhere, given a bound on the contexts so wide that the
choice falls on it, and windows over enough rows.  Against the 64-bit
definition within the bounds of kv_ref.check."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
ERR_PAGE = 0x8
# query rows x 64-key tiles above which a call is much work
WORK = 1200 * 152


def widen(table, rows):
    """The table with as many columns as make a call of `rows` rows (over all
    sequences and key heads) much work, and the bound on its contexts."""
    pages = max(WORK // rows + 1, table.shape[1])
    wide = torch.full((table.shape[0], pages), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide, pages * 64


def attend(q, cache, table, ctx, starts, qs, window=0, sinks=0, scale=None, max_q=None, **kw):
    max_q = max_q or max(qs)
    wide, bound = widen(table, len(ctx) * max_q * q.shape[1])
    return F().paged_attention_fp8(q, *cache, wide, A.i32(ctx), bound, q_starts=A.i32(starts),
                                   max_q=max_q, window=window, sinks=sinks, softmax_scale=scale,
                                   **kw)


def check(got, q, cache, table, ctx, starts, window=0, sinks=0, scale=None):
    D = q.shape[2]
    ref = R.dense(q, cache, table, ctx, starts, window, sinks, D ** -0.5 if scale is None else scale)
    R.check(got[0].view(-1, D), got[1].view(-1), ref, max(ctx) + 1)


@pytest.mark.parametrize("ctx,qs", [
    ([128], [128]), ([129], [129]), ([1], [1]), ([300], [40]), ([1000, 77], [64, 77]),
    ([513, 0, 640], [513, 0, 5]), ([2000], [33]), ([100, 40, 0], [160, 160, 160]),
    ([130, 55, 1, 700, 100, 640], [130, 0, 1, 257, 64, 3]), ([9000, 3, 700], [40, 40, 40])])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(66, 2, 128, BF), (40, 1, 64, HF), (132, 1, 128, HF),
                                            (260, 2, 64, BF)])
def test_prompts(ctx, qs, Hq, Hkv, D, dtype):
    q, cache, table, starts = A.setup(ctx, qs, Hq, Hkv, D, dtype, Hq + sum(ctx))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attend(q, cache, table, ctx, starts, qs, err_flags=err)
    check(got, q, cache, table, ctx, starts)
    assert int(err.item()) == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (130, 70), (129, 0), (600, 200)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(32, 2, 128, BF), (32, 4, 64, HF)])
def test_windows(window, sinks, Hq, Hkv, D, dtype):
    ctx, qs = [700, 1000, 450], [450, 449, 450]
    assert len(ctx) * max(qs) * Hq * min((window + max(qs)) // 64, 8) > WORK
    q, cache, table, starts = A.setup(ctx, qs, Hq, Hkv, D, dtype, window)
    got = F().paged_attention_fp8(q, *cache, table, A.i32(ctx), 1000, q_starts=A.i32(starts),
                                  max_q=450, window=window, sinks=sinks)
    check(got, q, cache, table, ctx, starts, window, sinks)


@pytest.mark.parametrize("mag,scale", [(30.0, None), (1e-30, 0.3), (1e-3, -0.5), (1.0, 0.0)])
def test_magnitudes_and_scales(mag, scale):
    ctx, qs, D = [333, 260], [64, 64], 128
    q, cache, table, starts = A.setup(ctx, qs, 8, 2, D, BF, 5)
    q = (q.float() * mag).to(BF)
    check(attend(q, cache, table, ctx, starts, qs, scale=scale), q, cache, table, ctx, starts,
          scale=scale)


def test_page_scales_far_apart():
    ctx, qs, D = [640, 300], [40, 40], 128
    q, cache, table, starts = A.setup(ctx, qs, 8, 2, D, BF, 3)
    kc, vc, ks, vs = cache
    for b, c in enumerate(ctx):
        for p in range((c + 63) // 64):
            page = int(table[b, p])
            if p % 3 == 1:
                vs[page] *= 2.0 ** (40 if b else -40)
            if p % 3 == 2:
                vc[page] = 0
                vs[page] = 2.0 ** -126
    check(attend(q, cache, table, ctx, starts, qs), q, cache, table, ctx, starts)


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_bad_pages(bad):
    ctx, D, n = [500], 128, 50
    q, cache, table, starts = A.setup(ctx, [n], 8, 2, D, BF, 32)
    t = table.clone()
    t[0, 3] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(q, cache, t, ctx, starts, [n], err_flags=err)
    assert int(err.item()) == ERR_PAGE
    idx = torch.full((n, 500), -1, dtype=torch.int32)
    for i in range(n):
        keep = [s for s in range(500 - n + i + 1) if s // 64 != 3]
        idx[i, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
    ref = R.sparse(q, cache, table, idx.cuda(), [0] * n, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, 501)


def test_tokens_behind_max_q_and_strided_queries():
    ctx, D = [400], 64
    q, cache, table, starts = A.setup(ctx, [200], 4, 2, D, BF, 31)
    packed = torch.randn(200, 9, D, device="cuda").to(BF)
    packed[:, 2:6] = q
    out = torch.full((200, 4, D), 3.0, dtype=BF, device="cuda")
    lse = torch.full((200, 4), 3.0, device="cuda")
    attend(packed[:, 2:6], cache, table, ctx, starts, [200], max_q=100, out=out, lse=lse)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    ref = tuple(x.view(200, 4, -1)[:100].reshape(-1, *x.shape[1:]) for x in ref)
    R.check(out[:100].reshape(-1, D), lse[:100].reshape(-1), ref, 401)
    assert bool((out[100:] == 3.0).all()) and bool((lse[100:] == 3.0).all())


def test_deterministic_and_captured():
    ctx, D = [3000, 2000], 128
    q, cache, table, starts = A.setup(ctx, [100, 90], 8, 2, D, BF, 41)
    wide, bound = widen(table, 2 * 100 * 8)
    args = (q, *cache, wide, A.i32(ctx), bound)
    kw = dict(q_starts=A.i32(starts), max_q=100)
    first = F().paged_attention_fp8(*args, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = F().paged_attention_fp8(*args, **kw)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("pages", [8, 48, 100])
def test_items_whole_and_cut(pages):
    """One sequence of long context among short ones: each bound on the
    contexts gives another share to the CTAs of the kernel for few rows."""
    ctx, D = [500, 3, 0, 77], 128
    q, cache, table, starts = A.setup(ctx, [1] * 4, 16, 2, D, BF, pages)
    wide = torch.full((4, pages), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    got = F().paged_attention_fp8(q, *cache, wide, A.i32(ctx), pages * 64)
    check(got, q, cache, table, ctx, starts)
