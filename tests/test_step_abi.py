"""CPU-only checks of include/fp4idx_step.h: exported symbols, the host-side
refusals of each call before anything touches CUDA, the binding's argument checks
and the stream that its allocations are made on."""
import contextlib
import ctypes
import os
import re
import subprocess
import types

import pytest
import torch

from tests import test_stream_argument as S


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
BIG = 1 << 40


@pytest.fixture(autouse=True)
def _no_visible_gpu(request):
    if "fake_ptr" in request.keywords and torch.cuda.is_available():
        pytest.skip("fake-pointer host-check tests run only where no GPU is visible")


def test_exports_every_declared_symbol(F):
    names = F.declared_symbols(F.STEP_HEADER_PATH)
    assert set(names) == {"fp4idx_batch_extend", "fp4idx_pages_release", "fp4idx_rope_qk",
                          "fp4idx_prompt_workspace_bytes", "fp4idx_prompt_attention"}
    out = subprocess.run(["nm", "-D", "--defined-only", F.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\bT (fp4idx_\w+)", out))


def test_constants_are_the_header_s(F):
    with open(F.STEP_HEADER_PATH) as f:
        text = f.read()
    assert int(re.search(r"FP4IDX_ERRFLAG_FULL (0x\w+)u", text).group(1), 16) == F.ERRFLAG_FULL
    assert f"FP4IDX_AXES_SECTIONS = {F.AXES_SECTIONS}" in text
    assert f"FP4IDX_AXES_INTERLEAVED = {F.AXES_INTERLEAVED}" in text


def call_extend(F, over):
    a = dict(cached=A[0], new=A[1], table=A[2], stride=20, pages=20, free=A[3], count=A[4], cap=50,
             starts=A[5], ctx=A[6], slots=A[7], pos=A[8], ids=A[9], lens=A[10], B=3, T=9, err=None)
    a.update(over)
    return F.lib().fp4idx_batch_extend(
        a["cached"], a["new"], a["table"], a["stride"], a["pages"], a["free"], a["count"], a["cap"],
        a["starts"], a["ctx"], a["slots"], a["pos"], a["ids"], a["lens"], a["B"], a["T"], a["err"],
        None)


POOL = [
    (dict(B=-1), "ERR_SHAPE"), (dict(B=1 << 31), "ERR_SHAPE"), (dict(stride=19), "ERR_SHAPE"),
    (dict(pages=-1), "ERR_SHAPE"), (dict(pages=1 << 25, stride=1 << 25), "ERR_SHAPE"),
    (dict(cap=-1), "ERR_SHAPE"), (dict(cap=1 << 31), "ERR_SHAPE"), (dict(stride=BIG), "ERR_SHAPE"),
    (dict(table=None), "ERR_NULL"), (dict(free=None), "ERR_NULL"), (dict(count=None), "ERR_NULL"),
    (dict(table=A[2] + 2), "ERR_ALIGN"), (dict(free=A[3] + 1), "ERR_ALIGN"),
    (dict(count=A[4] + 2), "ERR_ALIGN"), (dict(err=A[11] + 2), "ERR_ALIGN")]


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", POOL + [
    (dict(T=-1), "ERR_SHAPE"), (dict(T=1 << 31), "ERR_SHAPE"), (dict(cached=None), "ERR_NULL"),
    (dict(new=None), "ERR_NULL"), (dict(ctx=A[0]), "ERR_ARG"),
    (dict(ctx=A[1]), "ERR_ARG"), (dict(starts=A[0]), "ERR_ARG"), (dict(starts=A[1]), "ERR_ARG"),
    (dict(cached=A[0] + 2), "ERR_ALIGN"),
    (dict(new=A[1] + 2), "ERR_ALIGN"), (dict(starts=A[5] + 2), "ERR_ALIGN"),
    (dict(ctx=A[6] + 1), "ERR_ALIGN"), (dict(slots=A[7] + 4), "ERR_ALIGN"),
    (dict(pos=A[8] + 4), "ERR_ALIGN"), (dict(ids=A[9] + 2), "ERR_ALIGN"),
    (dict(lens=A[10] + 2), "ERR_ALIGN")], ids=str)
def test_extend_refusals(F, over, want):
    assert call_extend(F, over) == getattr(F, want)


def call_release(F, over):
    a = dict(held=A[0], kept=A[1], table=A[2], stride=20, pages=20, free=A[3], count=A[4], cap=50,
             B=3, err=None)
    a.update(over)
    return F.lib().fp4idx_pages_release(a["held"], a["kept"], a["table"], a["stride"], a["pages"],
                                        a["free"], a["count"], a["cap"], a["B"], a["err"], None)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", POOL + [
    (dict(held=None), "ERR_NULL"), (dict(kept=None), "ERR_NULL"),
    (dict(held=A[0] + 1), "ERR_ALIGN"), (dict(kept=A[1] + 2), "ERR_ALIGN")], ids=str)
def test_release_refusals(F, over, want):
    assert call_release(F, over) == getattr(F, want)


def call_rope(F, over):
    a = dict(q=A[0], qts=1024, qhs=128, qo=A[1], qots=1024, qohs=128, H=8, k=A[2], kts=256, khs=128,
             ko=A[3], kots=256, kohs=128, Hk=2, dt=0, D=128, pos=A[4], ps=5, sec=[16, 24, 24], n=3,
             order=0, cos=A[5], sin=A[6], max_pos=100, R=128, style=0, T=5, err=None)
    a.update(over)
    sec = (ctypes.c_int32 * len(a["sec"]))(*a["sec"]) if a["sec"] is not None else None
    return F.lib().fp4idx_rope_qk(
        a["q"], a["qts"], a["qhs"], a["qo"], a["qots"], a["qohs"], a["H"], a["k"], a["kts"],
        a["khs"], a["ko"], a["kots"], a["kohs"], a["Hk"], a["dt"], a["D"], a["pos"], a["ps"], sec,
        a["n"], a["order"], a["cos"], a["sin"], a["max_pos"], a["R"], a["style"], a["T"], a["err"],
        None)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", [
    (dict(T=-1), "ERR_SHAPE"), (dict(T=1 << 31), "ERR_SHAPE"), (dict(H=0), "ERR_SHAPE"),
    (dict(H=65536), "ERR_SHAPE"), (dict(Hk=-1), "ERR_SHAPE"), (dict(H=65535), "ERR_SHAPE"),
    (dict(D=8), "ERR_SHAPE"), (dict(D=132), "ERR_SHAPE"), (dict(D=1032), "ERR_SHAPE"),
    (dict(R=0), "ERR_SHAPE"), (dict(R=120), "ERR_SHAPE"), (dict(R=144), "ERR_SHAPE"),
    (dict(n=0), "ERR_SHAPE"), (dict(n=5), "ERR_SHAPE"), (dict(max_pos=0), "ERR_SHAPE"),
    (dict(q=None), "ERR_NULL"), (dict(qo=None), "ERR_NULL"), (dict(k=None), "ERR_NULL"),
    (dict(ko=None), "ERR_NULL"), (dict(pos=None), "ERR_NULL"), (dict(sec=None), "ERR_NULL"),
    (dict(cos=None), "ERR_NULL"), (dict(sin=None), "ERR_NULL"), (dict(dt=2), "ERR_ARG"),
    (dict(style=2), "ERR_ARG"), (dict(order=2), "ERR_ARG"), (dict(sec=[16, 24, 23]), "ERR_ARG"),
    (dict(sec=[-8, 48, 24]), "ERR_ARG"), (dict(sec=[64, 24, 24]), "ERR_ARG"),
    (dict(q=A[0] + 8), "ERR_ALIGN"), (dict(qo=A[1] + 8), "ERR_ALIGN"),
    (dict(k=A[2] + 2), "ERR_ALIGN"), (dict(ko=A[3] + 2), "ERR_ALIGN"), (dict(qts=1028), "ERR_ALIGN"),
    (dict(qhs=130), "ERR_ALIGN"), (dict(qots=1028), "ERR_ALIGN"), (dict(qohs=4), "ERR_ALIGN"),
    (dict(kts=260), "ERR_ALIGN"), (dict(khs=4), "ERR_ALIGN"), (dict(kots=260), "ERR_ALIGN"),
    (dict(kohs=4), "ERR_ALIGN"), (dict(pos=A[4] + 4), "ERR_ALIGN"), (dict(cos=A[5] + 8), "ERR_ALIGN"),
    (dict(sin=A[6] + 4), "ERR_ALIGN"), (dict(err=A[7] + 2), "ERR_ALIGN")], ids=str)
def test_rope_refusals(F, over, want):
    assert call_rope(F, over) == getattr(F, want)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over", [
    dict(qo=A[0], qots=2048), dict(qo=A[0], qohs=640), dict(ko=A[2], kots=512),
    dict(ko=A[2], kohs=640), dict(qo=A[0], qots=2048, T=5, k=None, Hk=0)], ids=str)
def test_rope_in_place_with_other_strides_is_refused(F, over):
    assert call_rope(F, over) == F.ERR_ARG


def call_prompt(F, over):
    a = dict(q=A[0], qts=1024, qhs=128, k=A[1], kts=256, khs=128, v=A[2], vts=256, vhs=128, dt=0,
             qs=A[3], ks=None, max_q=9, max_k=9, window=0, sinks=0, scale=0.1, out=A[4], lse=A[5],
             B=2, Tq=12, Tk=12, H=8, Hk=2, D=128, ws=A[6], wb=BIG, err=None)
    a.update(over)
    return F.lib().fp4idx_prompt_attention(
        a["q"], a["qts"], a["qhs"], a["k"], a["kts"], a["khs"], a["v"], a["vts"], a["vhs"], a["dt"],
        a["qs"], a["ks"], a["max_q"], a["max_k"], a["window"], a["sinks"], a["scale"], a["out"],
        a["lse"], a["B"], a["Tq"], a["Tk"], a["H"], a["Hk"], a["D"], a["ws"], a["wb"], a["err"],
        None)


@pytest.mark.fake_ptr
@pytest.mark.parametrize("over,want", [
    (dict(B=-1), "ERR_SHAPE"), (dict(Tq=-1), "ERR_SHAPE"), (dict(Tk=-1), "ERR_SHAPE"),
    (dict(H=7), "ERR_SHAPE"), (dict(H=0), "ERR_SHAPE"), (dict(Hk=0), "ERR_SHAPE"),
    (dict(H=1 << 20), "ERR_SHAPE"), (dict(Hk=65536, H=65536), "ERR_SHAPE"), (dict(D=96), "ERR_SHAPE"),
    (dict(max_q=0), "ERR_SHAPE"), (dict(max_q=1 << 29), "ERR_SHAPE"), (dict(max_k=-1), "ERR_SHAPE"),
    (dict(max_k=1 << 30), "ERR_SHAPE"), (dict(Tq=1 << 29), "ERR_SHAPE"),
    (dict(Tk=1 << 30), "ERR_SHAPE"), (dict(B=1 << 31), "ERR_SHAPE"),
    # rows that overlap: heads neither within a token's stride nor tokens in a head's
    (dict(kts=128, khs=128), "ERR_SHAPE"), (dict(vts=0), "ERR_SHAPE"), (dict(kts=-256), "ERR_SHAPE"),
    (dict(vts=128, vhs=11 * 128), "ERR_SHAPE"), (dict(kts=128, khs=12 * 128 + 8), "ERR_SHAPE"),
    (dict(kts=64), "ERR_SHAPE"), (dict(kts=1 << 34, khs=1 << 32), "ERR_SHAPE"),
    (dict(q=None), "ERR_NULL"), (dict(k=None), "ERR_NULL"), (dict(v=None), "ERR_NULL"),
    (dict(qs=None), "ERR_NULL"), (dict(out=None), "ERR_NULL"), (dict(ws=None), "ERR_NULL"),
    (dict(wb=1000), "ERR_SCRATCH"), (dict(dt=2), "ERR_ARG"), (dict(scale=-0.1), "ERR_ARG"),
    (dict(scale=float("nan")), "ERR_ARG"), (dict(scale=float("inf")), "ERR_ARG"),
    (dict(window=-1), "ERR_ARG"), (dict(sinks=-1), "ERR_ARG"), (dict(q=A[0] + 8), "ERR_ALIGN"),
    (dict(qts=1028), "ERR_ALIGN"), (dict(qhs=4), "ERR_ALIGN"), (dict(k=A[1] + 8), "ERR_ALIGN"),
    (dict(v=A[2] + 2), "ERR_ALIGN"), (dict(kts=260), "ERR_ALIGN"), (dict(vhs=124), "ERR_ALIGN"),
    (dict(out=A[4] + 8), "ERR_ALIGN"), (dict(lse=A[5] + 2), "ERR_ALIGN"),
    (dict(ws=A[6] + 8), "ERR_ALIGN"), (dict(qs=A[3] + 2), "ERR_ALIGN"),
    (dict(ks=A[7] + 2), "ERR_ALIGN"), (dict(err=A[8] + 2), "ERR_ALIGN")], ids=str)
def test_prompt_refusals(F, over, want):
    assert call_prompt(F, over) == getattr(F, want)


@pytest.mark.fake_ptr
def test_nothing_to_do_is_ok_without_touching_cuda(F):
    assert call_release(F, dict(B=0, held=None, kept=None)) == F.OK
    assert call_rope(F, dict(T=0, q=None)) == F.OK
    assert call_prompt(F, dict(Tq=0, q=None)) == F.OK
    assert call_prompt(F, dict(B=0, qs=None)) == F.OK


def test_workspace_bytes(F):
    n = F.prompt_workspace_bytes
    assert n(1, 1, 8, 1, 128) > n(1, 1, 8, 1, 64) > 0 and n(0, 1, 8, 1, 64) > 0
    for bad in ((-1, 1, 8, 1, 128), (1, 0, 8, 1, 128), (1, 1, 7, 2, 128), (1, 1, 0, 1, 64),
                (1, 1, 8, 0, 128), (1, 1, 8, 1, 80), (1 << 31, 1, 8, 1, 128), (1, 1 << 30, 8, 1, 64)):
        assert n(*bad) == 0, bad


def test_the_binding_refuses_what_it_cannot_pass_on(F, monkeypatch):
    """Host tensors, wrong types, shapes and devices raise before any call."""
    with pytest.raises(ValueError, match="CUDA"):
        i = torch.zeros(2, dtype=torch.int32)
        F.batch_extend(i, i, torch.zeros(2, 3, dtype=torch.int32), i, i[:1], 4)
    with pytest.raises(ValueError, match="CUDA"):
        F.rope_qk(torch.zeros(2, 1, 64).bfloat16(), None, torch.zeros(2).long(),
                  torch.zeros(4, 32), torch.zeros(4, 32))
    recorder = S.Recorder()
    monkeypatch.setattr(F, "_TORCH", recorder)
    monkeypatch.setattr(F, "_lib", S.Library(F._lib, recorder))
    g = S.gpu

    def i32(*shape):
        return g(torch.zeros(*shape, dtype=torch.int32))

    def bf(*shape):
        return g(torch.zeros(*shape, dtype=torch.bfloat16))

    pool = i32(3, 4), i32(9), i32(1)
    for bad in ((i32(2), i32(3), *pool), (i32(3), i32(4), *pool), (i32(3).long(), i32(3), *pool),
                (i32(3), g(torch.zeros(3)), *pool), (i32(3), i32(3), i32(12), *pool[1:]),
                (i32(3), i32(3), i32(4, 3).t(), *pool[1:]), (i32(3), i32(3), pool[0], i32(3, 3), pool[2]),
                (i32(3), i32(3), pool[0], pool[1], i32(2)), (i32(6)[::2], i32(3), *pool),
                (i32(3), i32(3), i32(4).expand(3, 4), *pool[1:]), (None, i32(3), *pool)):
        with pytest.raises((TypeError, ValueError)):
            F.batch_extend(*bad, 5)
        with pytest.raises((TypeError, ValueError)):
            F.pages_release(*bad)
    for bad in (dict(q_starts=i32(3)), dict(slot_mapping=i32(5)), dict(positions=g(torch.zeros(4).long())),
                dict(seq_ids=torch.zeros(5, dtype=torch.int32)), dict(row_lens=i32(10)[::2])):
        with pytest.raises((TypeError, ValueError)):
            F.batch_extend(i32(3), i32(3), *pool, 5, **bad)
    with pytest.raises(ValueError):
        F.batch_extend(i32(3), i32(3), *pool, -1)

    cos = g(torch.zeros(7, 32))
    pos, pos2 = g(torch.zeros(5).long()), g(torch.zeros(2, 5).long())
    q, k = bf(5, 4, 64), bf(5, 2, 64)
    for bad in ((q[..., :32], k, pos, cos, cos), (q.half(), k, pos, cos, cos), (q, k[:4], pos, cos, cos),
                (q[0], k, pos, cos, cos), (q, k, pos[:4], cos, cos), (q, k, pos.int(), cos, cos),
                (q, k, pos2, cos, cos), (q, k, pos, cos, cos[:6]), (q, k, pos, cos.t(), cos.t()),
                (q, k, pos, cos.double(), cos), (q.float(), None, pos, cos, cos),
                (q.transpose(1, 2), None, pos, cos, cos), (q, k, None, cos, cos)):
        with pytest.raises((TypeError, ValueError)):
            F.rope_qk(*bad)
    for bad in (dict(q_out=bf(5, 4, 32)), dict(q_out=bf(4, 4, 64)), dict(k_out=bf(5, 4, 64)),
                dict(q_out=g(torch.zeros(5, 4, 64))), dict(sections=[16, 16]),
                dict(rope_style="other")):
        with pytest.raises((TypeError, ValueError)):
            F.rope_qk(q, k, pos, cos, cos, **bad)
    with pytest.raises(ValueError):
        F.rope_qk(q, None, pos, cos, cos, k_out=k)

    st = i32(3)
    for bad in ((q, k, k[:4], st), (q, k, k.half(), st), (q, bf(5, 3, 64), bf(5, 3, 64), st),
                (q, bf(4, 2, 64), bf(4, 2, 64), st), (q, bf(5, 2, 128), bf(5, 2, 128), st),
                (q, k, k, st.long()), (q, k, k, i32(6)[::2]), (q, k, k, i32(0)), (q[0], k, k, st),
                (q, k[0], k[0], st)):
        with pytest.raises((TypeError, ValueError)):
            F.prompt_attention(*bad, 3)
    for bad in (dict(k_starts=st), dict(k_starts=i32(4), max_k=3), dict(out=bf(5, 4, 32)),
                dict(out=q.half()), dict(lse=g(torch.zeros(5, 2))), dict(workspace=i32(9)),
                dict(err_flags=g(torch.zeros(1)))):
        with pytest.raises((TypeError, ValueError)):
            F.prompt_attention(q, k, k, st, 3, **bad)
    assert recorder.ran == []


def test_allocations_are_made_on_the_stream_of_the_call(F, monkeypatch):
    recorder = S.Recorder()
    monkeypatch.setattr(F, "_TORCH", recorder)
    monkeypatch.setattr(F, "_lib", S.Library(F._lib, recorder))
    g, side = S.gpu, types.SimpleNamespace(cuda_stream=77)

    def i32(*shape):
        return g(torch.zeros(*shape, dtype=torch.int32))

    q, k = (g(torch.zeros(5, h, 64, dtype=torch.bfloat16)) for h in (4, 2))
    cos, pos = g(torch.zeros(7, 32)), g(torch.zeros(5).long())
    pool = i32(3, 4), i32(9), i32(1)
    for call in (lambda **kw: F.batch_extend(i32(3), i32(3), *pool, 5, **kw),
                 lambda **kw: F.batch_extend(i32(3), i32(3), *pool, 5, q_starts=i32(4), **kw),
                 lambda **kw: F.pages_release(i32(3), i32(3), *pool, **kw),
                 lambda **kw: F.rope_qk(q, k, pos, cos, cos, **kw),
                 lambda **kw: F.prompt_attention(q, k, k, i32(3), 3, **kw)):
        for s, want in ((None, 0), (side, 77)):
            recorder.made, recorder.ran = [], []
            call(**(dict(stream=s) if s else {}))
            assert set(recorder.made) <= {want} and recorder.ran == [want]
