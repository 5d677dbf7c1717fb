"""GPU tests of the token selection where the candidates come close to what fits
their list, whatever k: k on both sides of 1,024, rows as long as the bit map
allows.  Indices and counts exactly."""
import pytest
import torch

from tests.gpu_util import F

pytestmark = pytest.mark.gpu


def expect(x, k):
    """By value, ties from the lowest index up (a stable sort)."""
    at = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    return at.sort(dim=1).values.to(torch.int32)


@pytest.mark.parametrize("k", [1023, 1024, 1025, 1100, 1300, 1421, 1422, 1500, 2047, 2048, 3001,
                               4095, 4096])
@pytest.mark.parametrize("rows,cols", [(60, 65536), (25, 65537), (25, 131072), (12, 262144),
                                       (25, 16384)])
def test_every_k(rows, cols, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(cols + k)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    idx, cnt = F().topk_tokens(x, k)
    assert torch.equal(idx, expect(x, k)) and bool((cnt == k).all())
