"""GPU tests of the token selection over rows most of whose entries can never
be selected (-inf, NaN), with and without +inf among the rest: fewer samples
count than the threshold's rank asks for.  Indices and counts exactly."""
import pytest
import torch

from tests.test_topk_gpu import check

pytestmark = pytest.mark.gpu


def masked(rows, N, live, inf, seed):
    """A share `live` of the entries finite, a share `inf` of them +inf, the
    rest -inf and NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, N, generator=g, device="cuda")
    x = torch.where(torch.rand(rows, N, generator=g, device="cuda") < inf, float("inf"), x)
    dead = torch.rand(rows, N, generator=g, device="cuda")
    x = torch.where(dead >= live, -float("inf"), x)
    return torch.where(dead > 0.95, float("nan"), x)


@pytest.mark.parametrize("inf", [0.0, 0.003, 0.3, 1.0])
@pytest.mark.parametrize("live", [0.0, 1e-3, 0.02, 0.05, 0.1, 0.15, 0.2, 0.3, 0.4, 0.5])
@pytest.mark.parametrize("N,k", [(5000, 2048), (16384, 2048), (20001, 2048), (9300, 4096),
                                 (3301, 64), (3301, 1024)])
def test_few_live_entries(N, k, live, inf):
    check(masked(3, N, live, inf, N + k), k)


@pytest.mark.parametrize("rows", [1, 19, 20])
@pytest.mark.parametrize("live,inf", [(0.01, 0.0), (0.03, 0.5), (0.06, 0.01), (0.1, 0.0)])
def test_few_live_entries_of_long_rows(rows, live, inf):
    """Rows of a cluster each (up to 19), and of a CTA each."""
    lens = torch.tensor([[70003, 40000, 3500][i % 3] for i in range(rows)], dtype=torch.int32,
                        device="cuda")
    check(masked(rows, 70003, live, inf, rows), 1000, lens)


@pytest.mark.parametrize("cols", [4000, 16384])
@pytest.mark.parametrize("inf", [0.0, 0.01])
def test_prompt_rows_without_their_lengths(cols, inf):
    """A causal prompt's rows, -inf behind each token, after rows that left
    the CTAs' shared memory in every state."""
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    seen = torch.linspace(1, cols, 40, device="cuda").long()
    x = torch.randn(40, cols, generator=g, device="cuda")
    x = torch.where(torch.rand(40, cols, generator=g, device="cuda") < inf, float("inf"), x)
    x = torch.where(torch.arange(cols, device="cuda") < seen[:, None], x, -float("inf"))
    for _ in range(2):
        check(x, 1000)
        check(x.flip(1).contiguous(), 1000)
