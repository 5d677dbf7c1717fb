"""GPU tests of calls that the interface allows beside the usual ones: caches
that are parts of wider tensors, one tensor as keys and values, strided queries
and selections, table views, no lse, and non-finite keys and values in a store."""
import ctypes

import pytest
import torch

from tests import kv_ref as R
from tests import test_attention_gpu as A
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def relaid(cache, how):
    """The same cache as views of other tensors, poison around them."""
    kc, vc, ks, vs = cache
    B, H, n, D = kc.shape
    codes = torch.full((B + 2, 3, H + 1, n, D), 0x7F, dtype=torch.uint8, device="cuda")
    sc = torch.full((B + 2, 3, H + 1), float("nan"), device="cuda")
    codes[1:-1, 0, :H], codes[1:-1, 2, :H], sc[1:-1, 0, :H], sc[1:-1, 2, :H] = kc, vc, ks, vs
    view = [codes[1:-1, 0, :H], codes[1:-1, 2, :H], sc[1:-1, 0, :H], sc[1:-1, 2, :H]]
    if how == "fp8":
        view[:2] = [t.view(torch.float8_e4m3fn) for t in view[:2]]
    return view


def qview(q):
    """q as a view of a packed projection."""
    packed = torch.full((q.shape[0], q.shape[1] + 5, q.shape[2]), float("nan"), dtype=q.dtype,
                        device="cuda")
    packed[:, 2:2 + q.shape[1]] = q
    return packed[:, 2:2 + q.shape[1]]


def wide(table, cols):
    """The table as a view of as many columns as it has, of a wider tensor."""
    t = torch.full((table.shape[0], cols), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    t[:, 3:3 + table.shape[1]] = table
    return t[:, 3:3 + table.shape[1]]


@pytest.mark.parametrize("how", ["bytes", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,n", [(8, 2, 128, BF, 1), (6, 1, 64, HF, 3),
                                              (64, 2, 128, HF, 700), (64, 1, 64, BF, 700)])
def test_attention_over_parts_of_wider_tensors(Hq, Hkv, D, dtype, n, how):
    ctx = [1300, 800]
    q, cache, table, starts = A.setup(ctx, [n] * 2, Hq, Hkv, D, dtype, n + D)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = F().paged_attention_fp8(qview(q), *relaid(cache, how), wide(table, 40), A.i32(ctx),
                                       1300, err_flags=err)
    R.check(out.view(-1, D), lse.view(-1), ref, 1301)
    assert int(err.item()) == 0


@pytest.mark.parametrize("how", ["bytes", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, BF), (40, 1, 64, HF)])
def test_selection_over_parts_of_wider_tensors(Hq, Hkv, D, dtype, how):
    ctx = [1300, 800, 70]
    q, cache, table, _ = A.setup(ctx, [1] * 3, Hq, Hkv, D, dtype, D)
    table = table.clamp(min=0)
    idx = A.pick(A.gen(1), ctx, 3, 333)
    ref = R.sparse(q, cache, table, idx, [0, 1, 2], D ** -0.5)
    far = torch.full((3, 400), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    far[:, 9:342] = idx
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = F().sparse_attention_fp8(qview(q), *relaid(cache, how), wide(table, 40),
                                        far[:, 9:342], err_flags=err)
    R.check(out.view(-1, D), lse.view(-1), ref, 334)
    assert int(err.item()) == 0


@pytest.mark.parametrize("n", [1, 700])
def test_one_tensor_as_keys_and_values(n):
    ctx, D = [1000, 701], 128
    q, (kc, _, ks, _), table, starts = A.setup(ctx, [n] * 2, 64, 2, D, BF, 5)
    cache = (kc, kc, ks, ks)
    ref = R.dense(q, cache, table, ctx, starts, 0, 0, D ** -0.5)
    out, lse = F().paged_attention_fp8(q, *cache, table, A.i32(ctx), 1000)
    R.check(out.view(-1, D), lse.view(-1), ref, 1001)


@pytest.mark.parametrize("n", [1, 700])
def test_no_lse(n):
    """The C entry points without the optional outputs."""
    f = F()
    ctx, D, Hq, Hkv = [2000, 800], 128, 64, 2
    q, cache, table, _ = A.setup(ctx, [n] * 2, Hq, Hkv, D, BF, 6)
    table, lens = table.clamp(min=0), A.i32(ctx)
    want = f.paged_attention_fp8(q, *cache, table, lens, 2000)[0]
    idx = A.pick(A.gen(2), [800] * 2 * n, 2 * n, 200)
    picked = f.sparse_attention_fp8(q, *cache, table, idx)[0]
    c, _ = f._kv_cache(*cache)
    out = torch.zeros_like(q)
    ws = torch.empty(f.attention_workspace_bytes(2, n, Hq, Hkv, D), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert f.lib().fp4idx_paged_attention_fp8(
        q.data_ptr(), Hq * D, D, 0, ctypes.byref(c), table.data_ptr(), table.shape[1],
        lens.data_ptr(), None, 0, 2000, 0, 0, D ** -0.5, out.data_ptr(), None, 2, 2 * n, Hq,
        ws.data_ptr(), ws.numel(), None, s) == f.OK
    assert torch.equal(out, want)
    ws = torch.empty(f.attention_workspace_bytes(2 * n, 1, Hq, Hkv, D), dtype=torch.uint8,
                     device="cuda")
    assert f.lib().fp4idx_sparse_attention_fp8(
        q.data_ptr(), Hq * D, D, 0, ctypes.byref(c), table.data_ptr(), table.shape[1],
        table.shape[1], None, idx.data_ptr(), 200, 200, D ** -0.5, out.data_ptr(), None, 2, 2 * n,
        Hq, ws.data_ptr(), ws.numel(), None, s) == f.OK
    assert torch.equal(out, picked)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [1, 5, 64])
def test_store_of_values_that_are_not_finite(rows, dtype):
    """NaN leaves the scale to the others and is stored as NaN; an infinity
    makes the scale 2^127 and the largest code."""
    H, D = 3, 64
    g = A.gen(rows)
    cache = [torch.zeros(4, H, 64, D, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.ones(4, H, device="cuda") for _ in range(2)]
    x = torch.randn(rows, H, D, generator=g, device="cuda").to(dtype)
    y = x.clone()
    nan = torch.rand(rows, H, D, generator=g, device="cuda") < 0.3
    x[nan] = float("nan")
    x[:, 1] = float("nan")  # a head of NaN alone: amax 0
    y[rows // 2, 0, 7], y[0, 2, 3] = float("inf"), -float("inf")
    F().kv_store_fp8(x, y, torch.arange(rows, device="cuda") + 64, *cache)
    kc, vc, ks, vs = (t[1] for t in cache)
    keep = torch.where(x.isnan(), 0.0, x.double())
    want = R.block_scale(keep.abs().amax((0, 2)))
    assert torch.equal(ks.double(), want)
    got = R.codes_value(kc[:, :rows]).transpose(0, 1)
    assert torch.equal(got.isnan(), x.isnan())
    exact = R.e4m3_round(keep / want[None, :, None])
    assert torch.equal(torch.where(got.isnan(), 0.0, got), torch.where(x.isnan(), 0.0, exact))
    assert vs[0] == vs[2] == 2.0 ** 127
    got = R.codes_value(vc[:, :rows]).transpose(0, 1)
    assert float(got[rows // 2, 0, 7]) == 448 and float(got[0, 2, 3]) == -448
    y[rows // 2, 0, 7] = y[0, 2, 3] = 0
    assert bool((got[:, 0].abs() + got[:, 2].abs()).sum() == 448 * 2)
    want = R.block_scale(y[:, 1].double().abs().amax())
    assert float(vs[1]) == float(want)
    assert torch.equal(got[:, 1], R.e4m3_round(y[:, 1].double() / want))
