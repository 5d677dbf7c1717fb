"""GPU tests of attention over block tables without columns: no sequence has a
cached token, so every output row is 0 and every lse -inf."""
import pytest
import torch

from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
ERR_PAGE = 0x8


def empty(got):
    return bool((got[0] == 0).all()) and bool(torch.isneginf(got[1]).all())


# 7,000 tokens x 32 heads: the kernel for many rows
@pytest.mark.parametrize("batch,n", [(1, 1), (3, 4), (1, 7000)])
@pytest.mark.parametrize("D", [64, 128])
def test_no_context(batch, n, D):
    q, cache, _, _ = A.setup([64], [batch * n], 32, 2, D, torch.bfloat16, 1)
    table = torch.empty(batch, 0, dtype=torch.int32, device="cuda")
    for lens in ([0] * batch, [5] * batch):  # taken within the bound, 0
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for window in (0, 3):
            assert empty(F().paged_attention_fp8(q, *cache, table, A.i32(lens), 0, window=window,
                                                 err_flags=err))
        assert int(err.item()) == 0


def test_nothing_to_select():
    q, cache, _, _ = A.setup([64], [3], 8, 2, 128, torch.bfloat16, 2)
    table = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    none = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    assert empty(F().sparse_attention_fp8(q, *cache, table, none, err_flags=err))
    assert empty(F().sparse_attention_fp8(q, *cache, table, none[:, :0], err_flags=err))
    assert int(err.item()) == 0
    assert empty(F().sparse_attention_fp8(q, *cache, table, none + 1, err_flags=err))
    assert int(err.item()) == ERR_PAGE  # an entry behind a table of no pages
