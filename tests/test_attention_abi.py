"""CPU-only checks of include/fp4idx_attention.h: exported symbols, the
host-side refusals of each call before anything touches CUDA, and the
binding's argument checks."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def F():
    from fp4_sparse_attention_fp4idx_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from fp4_sparse_attention_fp4idx_gb300 import fp4idx
    return fp4idx


# Fake, aligned "device pointers", only ever passed with a defect that the
# host checks reject; and never where a CUDA device is visible.
A = [0x100000 * (i + 1) for i in range(20)]


@pytest.fixture(autouse=True)
def _no_visible_gpu(request):
    if "fake_ptr" in request.keywords and torch.cuda.is_available():
        pytest.skip("fake-pointer host-check tests run only where no GPU is visible")


def test_exports_every_declared_symbol(F):
    names = F.declared_symbols(F.ATTENTION_HEADER_PATH)
    assert set(names) == {"fp4idx_kv_store_fp8", "fp4idx_kv_load_fp8",
                          "fp4idx_attention_workspace_bytes", "fp4idx_paged_attention_fp8",
                          "fp4idx_sparse_attention_fp8", "fp4idx_topk_tokens"}
    out = subprocess.run(["nm", "-D", "--defined-only", F.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\bT (fp4idx_\w+)", out))


def test_the_cache_block_has_the_header_s_layout(F):
    with open(F.ATTENTION_HEADER_PATH) as f:
        body = re.search(r"typedef struct fp4idx_kv_cache \{(.*?)\}", f.read(), re.S).group(1)
    fields = re.findall(r"(\w+)(\*?) (\w+);", body)
    assert [n for _, _, n in fields] == [n for n, _ in F.KvCache._fields_]
    size = {"int64_t": 8, "int32_t": 4}
    assert ctypes.sizeof(F.KvCache) == sum(8 if p else size[t] for t, p, _ in fields)


CACHE = dict(kc=A[0], vc=A[1], ks=A[2], vs=A[3], blocks=10, cstride=2 * 64 * 128, sstride=2,
             heads=2, dim=128)


def cache_of(F, over):
    c = dict(CACHE)
    c.update({k: v for k, v in over.items() if k in c})
    return F.KvCache(c["kc"], c["vc"], c["ks"], c["vs"], c["blocks"], c["cstride"], c["sstride"],
                     c["heads"], c["dim"])


CACHE_DEFECTS = [
    (dict(kc=None), "ERR_NULL"), (dict(vc=None), "ERR_NULL"), (dict(ks=None), "ERR_NULL"),
    (dict(vs=None), "ERR_NULL"), (dict(blocks=0), "ERR_SHAPE"), (dict(blocks=1 << 31), "ERR_SHAPE"),
    (dict(cstride=2 * 64 * 128 - 16), "ERR_SHAPE"), (dict(cstride=1 << 62), "ERR_SHAPE"),
    (dict(cstride=2 * 64 * 128 + 8), "ERR_ALIGN"), (dict(sstride=1), "ERR_SHAPE"),
    (dict(heads=0), "ERR_SHAPE"), (dict(heads=65536, sstride=1 << 20, cstride=1 << 30), "ERR_SHAPE"),
    (dict(dim=96), "ERR_SHAPE"), (dict(kc=A[0] + 8), "ERR_ALIGN"), (dict(vs=A[3] + 2), "ERR_ALIGN"),
]


def call_store(F, over):
    a = dict(k=A[4], v=A[5], kts=256, khs=128, vts=256, vhs=128, dt=0, slots=A[6], T=4, err=None)
    a.update({k: v for k, v in over.items() if k in a})
    c = cache_of(F, over)
    return F.lib().fp4idx_kv_store_fp8(a["k"], a["v"], a["kts"], a["khs"], a["vts"], a["vhs"],
                                       a["dt"], a["slots"], None if "cache" in over else
                                       ctypes.byref(c), a["T"], a["err"], None)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", CACHE_DEFECTS + [
    (dict(cache=None), "ERR_NULL"), (dict(T=-1), "ERR_SHAPE"), (dict(T=1 << 31), "ERR_SHAPE"),
    (dict(k=None), "ERR_NULL"), (dict(v=None), "ERR_NULL"), (dict(slots=None), "ERR_NULL"),
    (dict(dt=2), "ERR_ARG"), (dict(dt=-1), "ERR_ARG"), (dict(k=A[4] + 8), "ERR_ALIGN"),
    (dict(v=A[5] + 2), "ERR_ALIGN"), (dict(kts=260), "ERR_ALIGN"), (dict(khs=132), "ERR_ALIGN"),
    (dict(vts=257), "ERR_ALIGN"), (dict(vhs=4), "ERR_ALIGN"), (dict(slots=A[6] + 4), "ERR_ALIGN"),
    (dict(err=A[7] + 1), "ERR_ALIGN")], ids=str)
def test_store_refusals(F, over, want):
    assert call_store(F, over) == getattr(F, want)


def call_load(F, over):
    a = dict(ko=A[4], vo=A[5], dt=1, slots=A[6], T=4, err=None)
    a.update({k: v for k, v in over.items() if k in a})
    c = cache_of(F, over)
    return F.lib().fp4idx_kv_load_fp8(None if "cache" in over else ctypes.byref(c), a["slots"],
                                      a["ko"], a["vo"], a["dt"], a["T"], a["err"], None)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", CACHE_DEFECTS + [
    (dict(cache=None), "ERR_NULL"), (dict(T=-1), "ERR_SHAPE"), (dict(ko=None), "ERR_NULL"),
    (dict(vo=None), "ERR_NULL"), (dict(slots=None), "ERR_NULL"), (dict(dt=7), "ERR_ARG"),
    (dict(ko=A[4] + 8), "ERR_ALIGN"), (dict(slots=A[6] + 4), "ERR_ALIGN"),
    (dict(err=A[7] + 2), "ERR_ALIGN")], ids=str)
def test_load_refusals(F, over, want):
    assert call_load(F, over) == getattr(F, want)


BIG = 1 << 40


def call_dense(F, over):
    a = dict(q=A[4], qts=8 * 128, qhs=128, dt=0, table=A[5], bts=16, ctx=A[6], starts=None, max_q=2,
             max_ctx=1000, window=0, sinks=0, scale=0.1, out=A[7], lse=A[8], batch=3, T=6, H=8,
             ws=A[9], wb=BIG, err=None)
    a.update({k: v for k, v in over.items() if k in a})
    c = cache_of(F, over)
    return F.lib().fp4idx_paged_attention_fp8(
        a["q"], a["qts"], a["qhs"], a["dt"], None if "cache" in over else ctypes.byref(c),
        a["table"], a["bts"], a["ctx"], a["starts"], a["max_q"], a["max_ctx"], a["window"],
        a["sinks"], a["scale"], a["out"], a["lse"], a["batch"], a["T"], a["H"], a["ws"], a["wb"],
        a["err"], None)


COMMON = CACHE_DEFECTS + [
    (dict(cache=None), "ERR_NULL"), (dict(q=None), "ERR_NULL"), (dict(table=None), "ERR_NULL"),
    (dict(out=None), "ERR_NULL"), (dict(ws=None), "ERR_NULL"), (dict(H=7), "ERR_SHAPE"),
    (dict(H=0), "ERR_SHAPE"), (dict(H=1 << 21), "ERR_SHAPE"), (dict(T=-1), "ERR_SHAPE"),
    (dict(batch=-1), "ERR_SHAPE"), (dict(batch=0), "ERR_SHAPE"), (dict(wb=1000), "ERR_SCRATCH"),
    (dict(dt=3), "ERR_ARG"), (dict(scale=float("nan")), "ERR_ARG"),
    (dict(scale=float("inf")), "ERR_ARG"), (dict(q=A[4] + 2), "ERR_ALIGN"),
    (dict(qts=1028), "ERR_ALIGN"), (dict(qhs=130), "ERR_ALIGN"), (dict(table=A[5] + 1), "ERR_ALIGN"),
    (dict(out=A[7] + 8), "ERR_ALIGN"), (dict(lse=A[8] + 2), "ERR_ALIGN"),
    (dict(ws=A[9] + 8), "ERR_ALIGN"), (dict(err=A[10] + 1), "ERR_ALIGN"),
]


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", COMMON + [
    (dict(ctx=None), "ERR_NULL"), (dict(T=7), "ERR_SHAPE"), (dict(max_ctx=-1), "ERR_SHAPE"),
    (dict(max_ctx=1025), "ERR_SHAPE"), (dict(max_ctx=1 << 30, bts=1 << 40), "ERR_SHAPE"),
    (dict(starts=A[11], max_q=0), "ERR_SHAPE"), (dict(starts=A[11], max_q=1 << 30), "ERR_SHAPE"),
    (dict(window=-1), "ERR_ARG"), (dict(sinks=-1), "ERR_ARG"), (dict(ctx=A[6] + 2), "ERR_ALIGN"),
    (dict(starts=A[11] + 2), "ERR_ALIGN")], ids=str)
def test_paged_attention_refusals(F, over, want):
    assert call_dense(F, over) == getattr(F, want)


def call_sparse(F, over):
    a = dict(q=A[4], qts=8 * 128, qhs=128, dt=0, table=A[5], bts=16, pages=16, seqs=None, idx=A[6],
             ids=64, n=64, scale=0.1, out=A[7], lse=A[8], batch=3, T=6, H=8, ws=A[9], wb=BIG,
             err=None)
    a.update({k: v for k, v in over.items() if k in a})
    c = cache_of(F, over)
    return F.lib().fp4idx_sparse_attention_fp8(
        a["q"], a["qts"], a["qhs"], a["dt"], None if "cache" in over else ctypes.byref(c),
        a["table"], a["bts"], a["pages"], a["seqs"], a["idx"], a["ids"], a["n"], a["scale"],
        a["out"], a["lse"], a["batch"], a["T"], a["H"], a["ws"], a["wb"], a["err"], None)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", COMMON + [
    (dict(idx=None), "ERR_NULL"), (dict(T=7), "ERR_SHAPE"), (dict(n=-1), "ERR_SHAPE"),
    (dict(n=65), "ERR_SHAPE"), (dict(n=1 << 30, ids=1 << 30), "ERR_SHAPE"),
    (dict(pages=-1), "ERR_SHAPE"), (dict(pages=17), "ERR_SHAPE"),
    (dict(pages=1 << 24, bts=1 << 24), "ERR_SHAPE"), (dict(idx=A[6] + 2), "ERR_ALIGN"),
    (dict(seqs=A[11] + 1), "ERR_ALIGN")], ids=str)
def test_sparse_attention_refusals(F, over, want):
    assert call_sparse(F, over) == getattr(F, want)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", [
    (dict(x=None), "ERR_NULL"), (dict(idx=None), "ERR_NULL"), (dict(R=-1), "ERR_SHAPE"),
    (dict(N=-1), "ERR_SHAPE"), (dict(R=1 << 31), "ERR_SHAPE"), (dict(N=1 << 30, xs=1 << 30), "ERR_SHAPE"),
    (dict(xs=99), "ERR_SHAPE"), (dict(k=0), "ERR_SHAPE"), (dict(k=4097, ids=5000), "ERR_SHAPE"),
    (dict(ids=63), "ERR_SHAPE"), (dict(x=A[0] + 2), "ERR_ALIGN"), (dict(idx=A[2] + 1), "ERR_ALIGN"),
    (dict(lens=A[1] + 2), "ERR_ALIGN"), (dict(cnt=A[3] + 2), "ERR_ALIGN")], ids=str)
def test_topk_refusals(F, over, want):
    a = dict(x=A[0], xs=100, lens=A[1], idx=A[2], ids=64, cnt=A[3], R=5, N=100, k=64)
    a.update(over)
    assert F.lib().fp4idx_topk_tokens(a["x"], a["xs"], a["lens"], a["idx"], a["ids"], a["cnt"],
                                      a["R"], a["N"], a["k"], None) == getattr(F, want)


@pytest.mark.fake_ptr
def test_nothing_to_do_is_ok_without_touching_cuda(F):
    assert call_store(F, dict(T=0, k=None, kc=None)) == F.OK
    assert call_load(F, dict(T=0, ko=None, cache=None)) == F.OK
    assert call_dense(F, dict(T=0, q=None)) == F.OK
    assert call_dense(F, dict(T=0, batch=0)) == F.OK
    assert call_sparse(F, dict(T=0, q=None)) == F.OK
    assert F.lib().fp4idx_topk_tokens(None, 0, None, None, 0, None, 0, 0, 0, None) == F.OK


def test_workspace_bytes(F):
    n = F.attention_workspace_bytes
    assert n(1, 1, 8, 1, 128) > 0 and n(4, 4, 32, 8, 64) % 256 == 0
    assert n(64, 1, 64, 8, 128) <= n(64, 4, 64, 8, 128)
    for bad in ((-1, 1, 8, 1, 128), (1, 0, 8, 1, 128), (1, 1, 7, 2, 128), (1, 1, 0, 1, 64),
                (1, 1, 8, 0, 128), (1, 1, 8, 1, 80), (1 << 31, 1, 8, 1, 128), (1, 1 << 30, 8, 1, 64),
                (1 << 20, 1 << 10, 32, 8, 128)):
        assert n(*bad) == 0, bad


def test_the_binding_refuses_what_it_cannot_pass_on(F):
    """Host tensors, wrong types and shapes raise before any call."""
    bf = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    codes, sc = torch.zeros(3, 1, 64, 64, dtype=torch.uint8), torch.zeros(3, 1)
    slots = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        F.kv_store_fp8(bf, bf, slots, codes, codes, sc, sc)
    with pytest.raises(TypeError, match="uint8"):
        F.kv_store_fp8(bf, bf, slots, codes.float(), codes, sc, sc)
    with pytest.raises(ValueError, match="CUDA"):
        F.topk_tokens(torch.zeros(2, 3), 1)
    with pytest.raises(TypeError, match="float32"):
        F.topk_tokens(torch.zeros(2, 3, dtype=torch.float64), 1)
    with pytest.raises(TypeError, match="torch.Tensor"):
        F.paged_attention_fp8(bf, None, codes, sc, sc, slots, slots, 5)
