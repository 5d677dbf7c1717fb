"""GPU tests of attention over values near the ends of the scales' range (a
page's scale goes down to 2^-126): the output follows the definition as long as
bf16 holds it, whole and joined from parts, for every form."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests import test_attention_tiles_gpu as T
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
RANGE = [-119, -116, -113, -110, -100, 100, 115]


def scaled(ctx, qs, Hq, Hkv, D, exp):
    q, cache, table, starts = A.setup(ctx, qs, Hq, Hkv, D, BF, 7 + D)
    cache[3].mul_(2.0 ** exp).clamp_(min=2.0 ** -126)
    assert bool(torch.isfinite(cache[3]).all())
    return q, cache, table, starts


@pytest.mark.parametrize("exp", RANGE)
@pytest.mark.parametrize("ctx", [[640, 300], [9000, 30]])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (32, 4, 64)])
def test_few_rows(ctx, Hq, Hkv, D, exp):
    q, cache, table, starts = scaled(ctx, [2, 2], Hq, Hkv, D, exp)
    out, lse = F().paged_attention_fp8(q, *cache, table, A.i32(ctx), max(ctx))
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, max(ctx) + 1)


@pytest.mark.parametrize("exp", RANGE)
@pytest.mark.parametrize("D", [128, 64])
def test_many_rows(D, exp):
    ctx, qs = [1640, 300], [200, 40]
    q, cache, table, starts = scaled(ctx, qs, 16, 2, D, exp)
    got = T.attend(q, cache, table, ctx, starts, qs)
    T.check(got, q, cache, table, ctx, starts)


@pytest.mark.parametrize("exp", RANGE)
@pytest.mark.parametrize("tokens,k", [(3, 200), (3, 2048)])
def test_selected_tokens(tokens, k, exp):
    ctx, D = [2500] * tokens, 128
    q, cache, table, _ = scaled(ctx, [1] * tokens, 16, 2, D, exp)
    idx = A.pick(A.gen(k), ctx, tokens, k)
    out, lse = F().sparse_attention_fp8(q, *cache, table, idx)
    ref = R.sparse(q, cache, table, idx, list(range(tokens)), D ** -0.5)
    R.check(out.view(-1, D), lse.view(-1), ref, k + 1)
