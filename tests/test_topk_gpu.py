"""GPU tests of the token selection against sorting: indices and counts
exactly."""
import pytest
import torch

from tests import kv_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu


def check(x, k, lens=None):
    ind, cnt = F().topk_tokens(x, k, row_lens=lens)
    n = lens.cpu().tolist() if lens is not None else [x.shape[1]] * x.shape[0]
    wi, wc = R.topk(x, k, n)
    assert torch.equal(cnt.cpu(), wc)
    assert torch.equal(ind.cpu(), wi)


def make(kind, R_, N, g):
    x = torch.randn(R_, N, generator=g, device="cuda")
    if kind == "ties":
        x = torch.round(x * 2) / 2
    elif kind == "equal":
        x = torch.full_like(x, -3.25)
    elif kind == "zeros":
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "holes":  # -inf, NaN of either sign, inf
        u = torch.rand(R_, N, generator=g, device="cuda")
        x = torch.where(u < 0.4, -float("inf"), x)
        x = torch.where(u > 0.8, float("nan"), x)
        x = torch.where((u > 0.9), -torch.full_like(x, float("nan")), x)
        x = torch.where((u > 0.4) & (u < 0.42), float("inf"), x)
    elif kind == "negative":
        x = -x.abs() - 1e-20
    elif kind == "tiny":
        x = x * 1e-42  # subnormals
    elif kind == "wide":
        x = x * torch.exp2(torch.randint(-100, 100, (R_, N), generator=g, device="cuda").float())
    elif kind == "rising":
        x = torch.arange(N, device="cuda").float().expand(R_, N).contiguous()
    elif kind == "falling":
        x = -torch.arange(N, device="cuda").float().expand(R_, N).contiguous()
    elif kind == "outliers":  # few large ones, the rest close together
        x = 1.0 + x * 1e-6
        x[:, ::97] += 100
    return x


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "zeros", "holes", "negative", "tiny",
                                  "wide", "rising", "falling", "outliers"])
@pytest.mark.parametrize("N,k", [(1, 1), (5, 64), (64, 64), (1025, 64), (5000, 2048), (20001, 2048),
                                 (40000, 333)])
def test_topk(kind, N, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + k)
    check(make(kind, 3, N, g), k)


@pytest.mark.parametrize("k", [1, 500, 4096])
def test_row_lengths(k):
    """Lengths of zero, one, below k, out of range, and NaN behind them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    lens = torch.tensor([0, 1, 2, 499, 500, 501, 4095, 4096, 4097, 9001, 20000, -5], device="cuda",
                        dtype=torch.int32)
    x = torch.randn(len(lens), 9001, generator=g, device="cuda")
    for r, n in enumerate(lens.tolist()):
        x[r, max(n, 0):] = float("nan")
    check(x, k, lens)


def test_rows_of_a_wider_matrix_and_a_given_output():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    big = torch.randn(6, 3001, generator=g, device="cuda")
    x = big[:, 1:2998]  # rows 4-byte aligned only
    check(x, 100)
    out = torch.full((6, 120), 77, dtype=torch.int32, device="cuda")
    F().topk_tokens(x, 100, indices=out[:, :100])
    wi, _ = R.topk(x, 100, [x.shape[1]] * 6)
    assert torch.equal(out[:, :100].cpu(), wi) and bool((out[:, 100:] == 77).all())


def test_many_rows_and_a_long_row():
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    check(torch.randn(700, 130, generator=g, device="cuda"), 64)
    check(torch.randn(1, 300007, generator=g, device="cuda"), 2048)
    check(torch.sort(torch.randn(2, 70001, generator=g, device="cuda")).values, 2048)


@pytest.mark.parametrize("rows", [1, 19, 20])
@pytest.mark.parametrize("kind", ["plain", "equal", "ties", "holes", "outliers", "falling"])
def test_long_rows_on_both_sides_of_the_cluster_rule(rows, kind):
    """Up to 19 rows are filtered by a cluster each; ragged lengths, some too
    short for every CTA of the cluster to have a share."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    lens = torch.tensor([[70003, 0, 3, 25, 3071, 3073, 40000][i % 7] for i in range(rows)],
                        dtype=torch.int32, device="cuda")
    big = make(kind, rows, 70006, g)
    check(big[:, 1:70004], 1000, lens)


def test_wide_maps_and_many_ties():
    """More columns than the histograms' memory holds a bit map for."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn(25, 140003, generator=g, device="cuda")
    x[:, ::50] = 3.0  # 2,801 equal ones near the border
    check(x, 2048)
    check(x[:3], 2048)


def test_empty():
    ind, cnt = F().topk_tokens(torch.empty(3, 0, device="cuda"), 8)
    assert bool((ind == -1).all()) and bool((cnt == 0).all())
    ind, cnt = F().topk_tokens(torch.empty(0, 9, device="cuda"), 8)
    assert ind.shape == (0, 8)
