"""CPU-only checks of limits that include/fp4idx_step.h states: refused by the host
checks of a call, before anything touches CUDA."""
import os

import pytest
import torch

from tests import test_step_abi as A


@pytest.fixture(scope="module")
def F():
    from fp4_sparse_attention_fp4idx_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from fp4_sparse_attention_fp4idx_gb300 import fp4idx
    return fp4idx


# Fake pointers, only ever passed with a defect that the host checks reject.
@pytest.fixture(autouse=True)
def _no_visible_gpu():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer host-check tests run only where no GPU is visible")


def header(F):
    with open(F.STEP_HEADER_PATH) as f:
        return " ".join(f.read().replace("\n *", " ").split())


@pytest.mark.parametrize("T,H,Hk,D,R", [
    (1 << 29, 1, 0, 128, 128), ((1 << 29) - 32, 8, 0, 128, 128), ((1 << 31) - 1, 1, 0, 32, 32),
    (1 << 26, 56, 8, 128, 64), ((1 << 32) // (64 * 8192), 65000, 535, 1024, 16)])
def test_rope_of_more_threads_than_a_grid_counts_is_refused(F, T, H, Hk, D, R):
    assert T * -(-D // 16) * -(-(H + Hk) // 8) >= (1 << 32) - 256
    k = dict(k=None) if Hk == 0 else dict(kts=Hk * D, khs=D, kots=Hk * D, kohs=D)
    assert A.call_rope(F, dict(T=T, H=H, Hk=Hk, D=D, R=R, n=1, sec=[R // 2], qts=H * D, qhs=D,
                               qots=H * D, qohs=D, **k)) == F.ERR_SHAPE
    assert "num_tokens * ceil(head_dim / 16) * ceil((q_heads + k_heads) / 8) below 2^32 - 256" \
        in header(F)
