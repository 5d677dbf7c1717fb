"""GPU tests of windowed attention over a cache whose pages out of sight are
gone: table entries of pages that hold no visible key are invalid or point to a
page of NaN, and the rows of visible pages that no query of the sequence sees
hold NaN codes.  None of them is looked up, flagged or used, by either kernel."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
WORK = 1200 * 152  # query rows x 64-key tiles above which a call is much work


def hide(cache, table, ctx, qs, window, sinks, gone):
    """Copies of the cache and the table in which everything that no query of a
    sequence sees is gone (`gone`: what the table says of its pages), and the
    number of hidden pages."""
    cache = [torch.cat([t, t[:1]]) for t in cache]  # the last block: the page of NaN
    kc, vc, ks, vs = cache
    kc[-1], vc[-1], ks[-1], vs[-1] = R.NAN_CODE, 0xFF, float("nan"), float("nan")
    table, hidden = table.clone(), 0
    for b, (c, n) in enumerate(zip(ctx, qs)):
        at = torch.arange((c + 63) // 64 * 64, device="cuda")
        unseen = (at >= c) | ((at <= c - n - window) & (at >= sinks)) | torch.tensor(n == 0).cuda()
        for p, rows in enumerate(unseen.view(-1, 64)):
            if bool(rows.all()):
                table[b, p] = -1 if gone == "invalid" else len(kc) - 1
                hidden += 1
            else:
                page = int(table[b, p])
                kc[page, :, rows], vc[page, :, rows] = 0xFF, R.NAN_CODE
    return cache, table, hidden


def run(ctx, qs, window, sinks, Hq, Hkv, D, dtype, gone):
    q, cache, table, starts = A.setup(ctx, qs, Hq, Hkv, D, dtype, window + sinks)
    ref = R.dense(q, cache, table, ctx, starts, window, sinks, D ** -0.5)
    cache, table, hidden = hide(cache, table, ctx, qs, window, sinks, gone)
    assert hidden > 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = F().paged_attention_fp8(q, *cache, table, A.i32(ctx), max(ctx),
                                       q_starts=A.i32(starts), max_q=max(qs), window=window,
                                       sinks=sinks, err_flags=err)
    R.check(out.view(-1, D), lse.view(-1), ref, max(ctx) + 1)
    assert int(err.item()) == 0


# 1,153 - 150 - 300 + 1 = 704, on a page's border in the first half of a
# 128-key tile; 640 + 64, in the second; the rest inside pages
CTX = [1153, 1089, 1999, 2000, 905, 150]


@pytest.mark.parametrize("gone", ["invalid", "nan"])
@pytest.mark.parametrize("window,sinks", [(300, 0), (300, 4), (236, 64), (511, 70), (385, 130)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(64, 2, 128, BF), (64, 4, 64, HF)])
def test_prompts(window, sinks, Hq, Hkv, D, dtype, gone):
    qs = [150, 150, 33, 149, 1, 150]
    tiles = min((window + 150) // 64, (max(CTX) + 63) // 64)
    assert len(CTX) * 150 * Hq * tiles > WORK  # the kernel for many rows
    run(CTX, qs, window, sinks, Hq, Hkv, D, dtype, gone)


@pytest.mark.parametrize("gone", ["invalid", "nan"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (300, 4), (236, 64), (129, 70)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 1, 128, BF), (32, 4, 64, HF), (16, 1, 128, HF)])
@pytest.mark.parametrize("n", [1, 4])
def test_drafted_tokens(n, window, sinks, Hq, Hkv, D, dtype, gone):
    run([1153, 1089, 700, 64, 0, 2000], [n] * 6, window, sinks, Hq, Hkv, D, dtype, gone)
