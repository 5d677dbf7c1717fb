"""CPU tests of the binding's check of block tables that are views: the bound
on the contexts must lie within the view's own columns, since what lies behind
them in its rows belongs to another tensor or to none.  The library is replaced
by a recorder; no CUDA call is made."""
import pytest
import torch

from tests.test_stream_argument import F, Library, Recorder, cache, gpu, ints  # noqa: F401


@pytest.fixture
def attend(F, monkeypatch):  # noqa: F811
    rec = Recorder()
    monkeypatch.setattr(F, "_TORCH", rec)
    monkeypatch.setattr(F, "_lib", Library(F.lib(), rec))

    def call(table, max_context, tokens=2):
        batch = table.shape[0]
        q = gpu(torch.zeros(tokens, 4, 64, dtype=torch.bfloat16))
        F.paged_attention_fp8(q, *cache(), table, ints(*[5] * batch), max_context)
        return len(rec.ran)

    call.error = F.Fp4idxError
    call.status = F.ERR_SHAPE
    return call


WIDE = torch.zeros(2, 10, dtype=torch.int32)


@pytest.mark.parametrize("table", [WIDE[:, :4], WIDE[:, 6:], WIDE[:1, :4], WIDE[:, 6:].contiguous()])
def test_a_bound_beyond_the_views_columns_is_refused(attend, table):
    for bad in (257, 300, 640):
        with pytest.raises(attend.error) as e:
            attend(gpu(table), bad)
        assert e.value.status == attend.status
    assert attend(gpu(table), 256) == 1
    assert attend(gpu(table), 1) == 2
    assert attend(gpu(table), 0) == 3


def test_a_call_without_tokens_has_no_bound(attend):
    attend(gpu(WIDE[:0]), 10 ** 6, tokens=0)
