"""GPU tests of attention for few rows with loose and tight bounds on the
contexts: the lengths decide on the device how the items are shared out, so
every bound gives the definition's result."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx", [[300] * 5, [64, 0, 9000, 1, 500], [6000], [0, 0], [2000] * 60,
                                 [(i * 397) % 3000 for i in range(90)]])
@pytest.mark.parametrize("Hq,Hkv,D,n", [(16, 2, 128, 1), (8, 8, 64, 2), (32, 4, 64, 4)])
def test_every_bound(ctx, Hq, Hkv, D, n):
    q, cache, table, starts = A.setup(ctx, [n] * len(ctx), Hq, Hkv, D, torch.bfloat16, len(ctx) + n)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    for pages in sorted({table.shape[1], table.shape[1] + 40, 2048}):
        wide = torch.full((len(ctx), pages), -7, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = F().paged_attention_fp8(q, *cache, wide, A.i32(ctx), pages * 64, err_flags=err)
        R.check(out.view(-1, D), lse.view(-1), ref, max(ctx) + 1)
        assert int(err.item()) == 0


def test_lengths_that_change_under_a_captured_call():
    """One graph, captured with a loose bound, over contexts that are cut and
    contexts that are not."""
    Hq, Hkv, D, B = 16, 2, 128, 6
    most = [9000, 500, 3, 700, 64, 2000]
    q, cache, table, starts = A.setup(most, [1] * B, Hq, Hkv, D, torch.bfloat16, 77)
    wide = torch.full((B, 1024), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    lens = A.i32(most)
    args = (q, *cache, wide, lens, 1024 * 64)
    F().paged_attention_fp8(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = F().paged_attention_fp8(*args)
    for ctx in (most, [100, 500, 3, 64, 0, 1], [0] * B, [9000, 1, 1, 1, 1, 1]):
        lens.copy_(A.i32(ctx))
        graph.replay()
        torch.cuda.synchronize()
        ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
        R.check(out.view(-1, D), lse.view(-1), ref, max(ctx) + 1)
