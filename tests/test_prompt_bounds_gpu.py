"""GPU tests that prompt_attention with starts out of order or out of range reads and
writes its tensors' rows only, and acts on the starts as they are taken."""
import pytest
import torch

from tests import step_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
T, PAD, MARK = 100, 70, 3.0


def inside(t, fill):
    """A copy of t inside a larger tensor that holds `fill` before and behind it."""
    whole = torch.full((t.shape[0] + 2 * PAD, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
    part = whole[PAD:PAD + t.shape[0]]
    part.copy_(t)
    return whole, part


CASES = [  # starts, what they are taken for, starts of the keys, what they are taken for
    ([-5, 100], [(0, 100)], None, None),
    ([0, 10 ** 9], [(0, 100)], None, None),
    ([-2 ** 31, 2 ** 31 - 1], [(0, 100)], None, None),
    ([90, 20, 100], [(90, 90), (20, 100)], None, None),
    ([2 ** 31 - 1, -2 ** 31, 7], [(100, 100), (0, 7)], None, None),
    ([40, 90, 60], [(40, 90), (90, 90)], None, None),
    ([5, 95], [(5, 95)], [60, 10 ** 9], [(60, 100)]),
    ([5, 95], [(5, 95)], [-7, 33], [(0, 33)]),
    ([0, 30, 60], [(0, 30), (30, 60)], [2 ** 31 - 1, 10, -4], [(100, 100), (10, 10)]),
    ([0, 30, 60], [(0, 30), (30, 60)], [50, 20, 10 ** 6], [(50, 50), (20, 100)])]


@pytest.mark.parametrize("starts,taken,kstarts,ktaken", CASES, ids=str)
@pytest.mark.parametrize("H,Hk,D,dtype,window", [
    (4, 2, 64, torch.bfloat16, 0), (6, 2, 128, torch.float16, 0), (8, 1, 128, torch.bfloat16, 20)])
def test_starts_are_taken_within_the_tensors(starts, taken, kstarts, ktaken, H, Hk, D, dtype,
                                             window):
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for h in (H, Hk, Hk))
    (_, q), (_, k), (_, v) = (inside(t, float("nan")) for t in (q, k, v))
    whole_out, out = inside(torch.full((T, H, D), MARK, device="cuda").to(dtype), MARK)
    whole_lse, lse = inside(torch.full((T, H), MARK, device="cuda"), MARK)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    F().prompt_attention(q, k, v, i32(starts), T, k_starts=None if kstarts is None else i32(kstarts),
                         max_k=T, window=window, out=out, lse=lse, err_flags=err)
    assert int(err) == 0
    left = torch.ones(T + 2 * PAD, dtype=torch.bool, device="cuda")
    for (a, b), (ka, kb) in zip(taken, ktaken or taken):
        if a == b:
            continue
        left[PAD + a:PAD + b] = False
        ref = R.attend(q[a:b], k[ka:kb], v[ka:kb], [0, b - a], [0, kb - ka], window, 0, D ** -0.5)
        R.check(out[a:b], lse[a:b], ref)
    assert bool((whole_out[left] == MARK).all()) and bool((whole_lse[left] == MARK).all())
