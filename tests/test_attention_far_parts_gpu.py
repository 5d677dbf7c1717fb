"""GPU tests of parts of one item whose weights and values lie far apart: a key
of weight e^-88 (below fp32's smallest normal) whose page's values are 2^122 times
as large counts by 2^-5, in whichever part of the cut item it falls."""
import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests import test_attention_tiles_gpu as T
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NEAR, FAR = 100, 6000  # positions of the two keys


def build(ctx, n, Hq, Hkv, D):
    """q = e_0, so that a key's first element is its score."""
    q, cache, table, starts = A.setup([ctx], [n], Hq, Hkv, D, BF, 11)
    q.zero_()
    q[..., 0] = 1
    kc, vc, ks, vs = cache
    kc.zero_()
    vc.zero_()
    ks.fill_(1)
    vs.fill_(1)
    code = {x: torch.tensor(float(x)).to(torch.float8_e4m3fn).view(torch.uint8).item()
            for x in (1, -88, -448)}
    kc[..., 0] = code[-448]
    for at, score, scale in ((NEAR, 0, 2.0 ** -89), (FAR, -88, 2.0 ** 33)):
        page = int(table[0, at // 64])
        kc[page, :, at % 64, 0] = code[score] if score else 0
        vc[page, :, at % 64] = code[1]
        vs[page] = scale
    return q, cache, table.clamp(min=0), starts


def check(got, ref, n):
    R.check(got[0].view(-1, got[0].shape[-1]), got[1].view(-1), ref, n)
    assert bool((got[0].double() > 2.0 ** -89 * (1 + 2.0 ** -6)).all())  # the far key counts


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (16, 2, 64)])
def test_few_rows(Hq, Hkv, D):
    q, cache, table, starts = build(9000, 1, Hq, Hkv, D)
    ref = R.dense(q, cache, table, [9000], starts, 0, 0, 1.0)
    check(F().paged_attention_fp8(q, *cache, table, A.i32([9000]), 9000, softmax_scale=1.0), ref,
          9001)


@pytest.mark.parametrize("D", [128, 64])
def test_many_rows(D):
    q, cache, table, starts = build(9000, 40, 32, 2, D)
    ref = R.dense(q, cache, table, [9000], starts, 0, 0, 1.0)
    check(T.attend(q, cache, table, [9000], starts, [40], scale=1.0), ref, 9001)


@pytest.mark.parametrize("D", [128, 64])
def test_selected_tokens(D):
    q, cache, table, _ = build(9000, 1, 16, 2, D)
    idx = torch.arange(2048, dtype=torch.int32, device="cuda")[None].clone()
    idx[0, 2000] = FAR
    ref = R.sparse(q, cache, table, idx, [0], 1.0)
    check(F().sparse_attention_fp8(q, *cache, table, idx, softmax_scale=1.0), ref, 2049)
