"""GPU tests of prompt_attention on bf16 values near the ends of their range, against
the 64-bit definition within the derived bounds (step_ref.check)."""
import pytest
import torch

from tests import step_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# one item of three tiles; items cut between CTAs and joined
SHAPES = [(300, 300, 64), (300, 300, 128), (1, 5000, 64), (1, 5000, 128), (3, 700, 128)]


def attend(scores, v, n):
    """n queries behind the others, whose scores with key s are scores[s], 4 heads
    over 2; out and lse held to the definition."""
    c, Hk, D = v.shape
    q = torch.zeros(n, 4, D, dtype=BF, device="cuda")
    q[..., 0] = 1
    k = torch.zeros(c, Hk, D, dtype=BF, device="cuda")
    k[..., 0] = scores.to(BF)[:, None]
    starts = [torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in (n, c)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = F().prompt_attention(q, k, v, starts[0], n, k_starts=starts[1], max_k=c,
                                    softmax_scale=1.0, err_flags=err)
    assert int(err) == 0
    assert bool(torch.isfinite(out).all())
    R.check(out, lse, R.attend(q, k, v, [0, n], [0, c], 0, 0, 1.0))


def values(c, D, top, seed):
    """Magnitudes of 2^(top - 1) to 2^top, signs at random."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = 0.5 + 0.49 * torch.rand(c, 2, D, generator=g, device="cuda", dtype=torch.float64)
    sign = torch.randint(0, 2, x.shape, generator=g, device="cuda") * 2 - 1
    return (x * sign * 2.0 ** top).to(BF)


@pytest.mark.parametrize("n,c,D", SHAPES)
@pytest.mark.parametrize("rise", [2.75, 5.5, 20.0])
def test_late_keys_of_large_weight_and_large_values(n, c, D, rise):
    """A score may exceed the reference of the row's sums by some powers of two before
    that moves; the sums stay finite all the same.  The magnitudes of the risers'
    values add up to less than 2^125, the others' are small."""
    scores = torch.zeros(c, device="cuda")
    scores[150::200] = rise
    risers = len(scores[150::200])
    v = values(c, D, 125 - (risers - 1).bit_length(), c + D)
    v[scores == 0] *= 2.0 ** -40
    attend(scores, v, n)


@pytest.mark.parametrize("n,c,D", SHAPES)
def test_equal_weights_up_to_the_bound(n, c, D):
    """The magnitudes of all of a row's values add up to less than 2^125."""
    attend(torch.zeros(c, device="cuda"), values(c, D, 125 - c.bit_length(), c).abs(), n)


@pytest.mark.parametrize("n,c,D", SHAPES)
def test_tiny_weights_of_large_values(n, c, D):
    """Keys of weight 2^-117 whose values make up half of the output."""
    scores = torch.full((c,), -200.0, device="cuda")
    scores[c // 2], scores[::7], scores[0] = 0.0, -81.0, 0.0
    v = values(c, D, 117 - (c // 7).bit_length(), 3)
    v[c // 2] = v[0] = 1.0
    attend(scores, v, n)


@pytest.mark.parametrize("n,c,D", SHAPES)
def test_small_values(n, c, D):
    attend(torch.linspace(-3, 3, c, device="cuda"), values(c, D, -100, 4), n)
