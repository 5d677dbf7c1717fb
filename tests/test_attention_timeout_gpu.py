"""The bounded waits' timeout path of both attention kernels on the GPU, without
a fault: the testing hook makes one launch leave out work of its first CTA, so
that CTA's waits run out after their 1 s limit.  That launch must return
normally with FP4IDX_ERRFLAG_TIMEOUT raised and nothing else, leave the rows of
other CTAs' items right, and the next launch must repeat the one before it."""
import time

import pytest
import torch

from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def run(call, n, index):
    f = F()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    f.test_withhold_next(f.TEST_ATTENTION, index)
    t0 = time.monotonic()
    got = call(err)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 10
    assert int(err.item()) == f.ERRFLAG_TIMEOUT
    # the last sequence's items are those of CTAs that had all their work
    assert torch.equal(got[0][-n:], want[0][-n:]) and torch.equal(got[1][-n:], want[1][-n:])
    err.zero_()
    again = call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_an_index_behind_the_work_withholds_nothing():
    f = F()
    q, cache, table, _ = A.setup([300], [1], 8, 2, 128, BF, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = A.i32([300])
    want = F().paged_attention_fp8(q, *cache, table, lens, 300)
    for index in (1000, 1 << 40):
        f.test_withhold_next(f.TEST_ATTENTION, index)
        got = f.paged_attention_fp8(q, *cache, table, lens, 300, err_flags=err)
        assert torch.equal(got[0], want[0])
    assert int(err.item()) == 0


@pytest.mark.parametrize("index", [0, 1, 6])  # the first rings' stages
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (32, 4, 64)])
def test_few_rows(Hq, Hkv, D, index):
    ctx = [20000, 9000, 300]
    q, cache, table, _ = A.setup(ctx, [1] * 3, Hq, Hkv, D, BF, 2)
    lens = A.i32(ctx)
    run(lambda err: F().paged_attention_fp8(q, *cache, table, lens, 20000, err_flags=err), 1,
        index)


@pytest.mark.parametrize("index", [0, 1])
def test_selected_tokens(index):
    ctx = [3000] * 40
    q, cache, table, _ = A.setup(ctx, [1] * 40, 16, 2, 128, BF, 3)
    idx = A.pick(A.gen(4), ctx, 40, 2048)
    run(lambda err: F().sparse_attention_fp8(q, *cache, table, idx, err_flags=err), 1, index)


@pytest.mark.parametrize("index", [0, 1, 11])
@pytest.mark.parametrize("D", [128, 64])
def test_many_rows(D, index):
    ctx = [6000, 5000]
    q, cache, table, starts = A.setup(ctx, [700, 300], 32, 2, D, BF, 5)
    lens, at = A.i32(ctx), A.i32(starts)
    assert 2 * 700 * 32 * (6000 // 64) > 1200 * 152  # the kernel for many rows
    run(lambda err: F().paged_attention_fp8(q, *cache, table, lens, 6000, q_starts=at, max_q=700,
                                            err_flags=err), 100, index)
