"""GPU test of prompt_attention on a batch of many places, most of them empty, beside a
long prompt: the result is that of the sequences alone, bit for bit."""
import pytest
import torch

from tests.gpu_util import F

pytestmark = pytest.mark.gpu


def starts(lens):
    x = torch.tensor([0, *lens], dtype=torch.int64)
    return x.cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("long,H,Hk,D,before,between", [
    (32768, 64, 1, 64, 5000, 30000),  # 8,192 row chunks in the long one
    (3000, 8, 2, 128, 31, 33), (3000, 8, 2, 128, 0, 32), (40, 32, 4, 64, 100, 1000)])
def test_empty_places_change_nothing(long, H, Hk, D, before, between):
    """A search that took an empty place's chunks one by one would let the waits for the
    next piece of work run out."""
    short = [1, 5, 0, 1, 300]
    full = [0] * before + [long] + [0] * between + short + [0] * between + [7] + [0] * 40
    lens = [n for n in full if n]
    g = torch.Generator(device="cuda")
    g.manual_seed(long)
    T = sum(lens)
    q = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(T, Hk, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    got = []
    for x in (lens, full):
        for window in (0, 500):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.full_like(q, float("nan"))
            got.append((*F().prompt_attention(q, k, v, starts(x), max(long, 300), window=window,
                                              out=out, err_flags=err), err))
    torch.cuda.synchronize()
    assert all(int(e) == 0 for *_, e in got)
    for a, b in zip(got[:2], got[2:]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(torch.isfinite(got[0][0]).all())


def test_one_long_chunk_and_hundreds_of_single_tokens():
    """Equal to the two kinds in calls of their own within the rounding of the output."""
    H, Hk, D, c = 8, 1, 128, 700
    qs = [1] * 128 + [2048] + [1] * 127
    ks = [c] * 128 + [2048] + [c] * 127
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randn(sum(qs), H, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(sum(ks), Hk, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, lse = F().prompt_attention(q, k, v, starts(qs), 2048, k_starts=starts(ks), max_k=2048)
    one, one_lse = F().prompt_attention(q[128:-127], k[128 * c:-127 * c], v[128 * c:-127 * c],
                                        starts([2048]), 2048)
    rows = torch.cat([torch.arange(128), torch.arange(128 + 2048, sum(qs))]).cuda()
    keys = torch.cat([torch.arange(128 * c), torch.arange(128 * c + 2048, sum(ks))]).cuda()
    single, single_lse = F().prompt_attention(q[rows], k[keys], v[keys], starts([1] * 255), 1,
                                              k_starts=starts([c] * 255), max_k=c)
    # an output is rounded by 2^-8 of itself and made from probabilities rounded as much,
    # in either call: 2 (2^-8 |o| + 2^-8 sum p |v|), with sum p |v| <= max |v|
    top = float(v.abs().max())
    for a, b in ((out[128:-127], one), (out[rows], single)):
        assert bool(((a - b).abs().float() <= 2.0 ** -7 * (b.abs().float() + top)).all())
    for a, b in ((lse[128:-127], one_lse), (lse[rows], single_lse)):
        assert float((a - b).abs().max()) < 2.0 ** -14
