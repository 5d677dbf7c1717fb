"""CPU tests of the binding's `stream` argument: whatever a call allocates is
allocated on the stream that its kernels run on, so that a fill is in order
with them and memory given back at the call's end is used again behind them
only.  The library and torch's allocations are replaced by recorders; no CUDA
call is made."""
import contextlib
import os
import types

import pytest
import torch


class OnGpu(torch.Tensor):
    """A host tensor that says it is on cuda:0."""

    def get_device(self):
        return 0

    is_cuda = property(lambda self: True)


def gpu(t):
    return t.as_subclass(OnGpu)


class Recorder:
    """torch, with the stream of each allocation noted."""

    def __init__(self):
        self.on, self.made, self.ran = None, [], []
        self.cuda = types.SimpleNamespace(
            stream=self._stream, current_stream=lambda *a: types.SimpleNamespace(cuda_stream=0),
            device=lambda *a: contextlib.nullcontext())
        self._C = types.SimpleNamespace(_cuda_getDevice=lambda: 0,
                                        _cuda_getCurrentRawStream=lambda dev: 0)

    def __getattr__(self, name):
        return getattr(torch, name)

    @contextlib.contextmanager
    def _stream(self, s):
        before, self.on = self.on, s
        yield
        self.on = before

    def _alloc(self, make, *args, **kw):
        self.made.append(self.on.cuda_stream if self.on is not None else 0)
        return gpu(make(*args, **kw))

    def empty(self, *args, **kw):
        return self._alloc(torch.empty, *args, **kw)

    def zeros(self, *args, **kw):
        return self._alloc(torch.zeros, *args, **kw)

    def empty_like(self, *args, **kw):
        return self._alloc(torch.empty_like, *args, **kw)


class Library:
    """The entry points, each of which notes the stream it is given."""

    def __init__(self, lib, recorder):
        self.lib, self.recorder = lib, recorder

    def __getattr__(self, name):
        if name.endswith(("_bytes", "_scale", "_string")):
            return getattr(self.lib, name)

        def call(*args):
            self.recorder.ran.append(getattr(args[-1], "value", args[-1]) or 0)
            return 0

        call.__name__ = name
        return call


@pytest.fixture
def F():
    from fp4_sparse_attention_fp4idx_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from fp4_sparse_attention_fp4idx_gb300 import fp4idx
    return fp4idx


SIDE = types.SimpleNamespace(cuda_stream=77)


def run(F, monkeypatch, call, made):
    """call(stream) allocates `made` buffers, all on the stream it runs on."""
    for stream in (None, SIDE):
        rec = Recorder()
        monkeypatch.setattr(F, "_TORCH", rec)
        monkeypatch.setattr(F, "_lib", Library(F.lib(), rec))
        call(stream)
        monkeypatch.undo()
        want = stream.cuda_stream if stream is not None else 0
        assert rec.ran == [want]
        assert rec.made == [want] * made, (stream, rec.made)


def cache(heads=2, dim=64):
    return [gpu(torch.zeros(4, heads, 64, dim, dtype=torch.uint8)) for _ in range(2)] + \
        [gpu(torch.ones(4, heads)) for _ in range(2)]


def ints(*v):
    return gpu(torch.tensor(v, dtype=torch.int32))


def test_load(F, monkeypatch):
    slots = gpu(torch.zeros(3, dtype=torch.int64))
    run(F, monkeypatch, lambda s: F.kv_load_fp8(*cache(), slots, stream=s), 2)
    one = gpu(torch.zeros(3, 2, 64, dtype=torch.bfloat16))
    run(F, monkeypatch, lambda s: F.kv_load_fp8(*cache(), slots, k_out=one, stream=s), 1)


def test_attention(F, monkeypatch):
    q = gpu(torch.zeros(2, 4, 64, dtype=torch.bfloat16))
    packed = gpu(torch.zeros(2, 6, 64, dtype=torch.bfloat16))[:, 1:5]
    table, lens = ints([0, 1], [2, 3]), ints(70, 5)
    for x in (q, packed):
        run(F, monkeypatch,
            lambda s: F.paged_attention_fp8(x, *cache(), table, lens, 128, stream=s), 3)
        run(F, monkeypatch,
            lambda s: F.sparse_attention_fp8(x, *cache(), table, ints([0, 65, -1], [1, 2, 3]),
                                             stream=s), 3)
    out, lse = gpu(torch.zeros_like(q)), gpu(torch.zeros(2, 4))
    run(F, monkeypatch, lambda s: F.paged_attention_fp8(q, *cache(), table, lens, 128, out=out,
                                                        lse=lse, stream=s), 1)


def test_topk(F, monkeypatch):
    x = gpu(torch.zeros(3, 50))
    run(F, monkeypatch, lambda s: F.topk_tokens(x, 8, stream=s), 2)
    run(F, monkeypatch, lambda s: F.topk_tokens(x, 1, counts=ints(0, 0, 0), stream=s), 1)


def bf(*shape):
    return gpu(torch.zeros(shape, dtype=torch.bfloat16))


def longs(n):
    return gpu(torch.zeros(n, dtype=torch.int64))


@pytest.mark.parametrize("hadamard", [False, True])
def test_prepass(F, monkeypatch, hadamard):
    cos = gpu(torch.zeros(9, 32))
    q, w, gamma = bf(2, 16, 128), bf(2, 16), bf(128)
    pages, pages8 = (gpu(torch.zeros(3, n, dtype=torch.uint8)) for n in (4352, 8448))
    kw = dict(hadamard=hadamard)
    run(F, monkeypatch, lambda s: F.q_rope_pack_weights(
        q, w, longs(2), cos, cos, stream=s, **kw), 3)
    run(F, monkeypatch, lambda s: F.indexer_prepass(
        bf(2, 128), gamma, longs(2), pages, q, w, longs(2), cos, cos, stream=s, **kw), 3)
    run(F, monkeypatch, lambda s: F.q_rope_fp8_weights(
        q, w, longs(2), cos, cos, stream=s, **kw), 2)
    run(F, monkeypatch, lambda s: F.indexer_prepass_fp8(
        bf(2, 128), gamma, longs(2), pages8, q, w, longs(2), cos, cos, stream=s, **kw), 2)


def test_scorers_and_fake_quant(F, monkeypatch):
    pages = gpu(torch.zeros(3, 4352, dtype=torch.uint8))
    q4, qs = (gpu(torch.zeros(2, 32, n, dtype=torch.uint8)) for n in (64, 4))
    wt = gpu(torch.zeros(2, 32))
    run(F, monkeypatch, lambda s: F.paged_mqa_logits(
        q4, qs, wt, pages, ints([0], [1]), ints(5, 6), 64, stream=s), 1)
    run(F, monkeypatch, lambda s: F.mqa_logits_prefill(
        q4, qs, wt, pages, ints(0, 0), ints(1, 2), 64, stream=s), 1)
    run(F, monkeypatch, lambda s: F.rope_fake_quant(
        bf(2, 128), longs(2), gpu(torch.zeros(9, 32)), gpu(torch.zeros(9, 32)), stream=s), 1)
