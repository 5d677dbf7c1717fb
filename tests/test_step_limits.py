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


@pytest.mark.parametrize("over", [
    # a broadcast tensor in place, or as an output: over the heads, over the tokens
    dict(q=A.A[0], qo=A.A[0], qts=128, qhs=0, qots=128, qohs=0), dict(qots=1024, qohs=0),
    dict(qots=0, qohs=128), dict(ko=A.A[2], kts=128, khs=0, kots=128, kohs=0),
    dict(kots=0, kohs=128),
    # rows, tokens or heads that reach into the next ones
    dict(qohs=120), dict(qots=128, qohs=128), dict(qots=1016), dict(qots=-1016, qohs=128),
    dict(qots=128, qohs=4 * 128 + 120), dict(H=1, qots=120), dict(T=1, qohs=64),
    dict(Hk=1, kots=64, kohs=128), dict(kots=256, kohs=-120)], ids=str)
def test_rope_outputs_whose_rows_overlap_are_refused(F, over):
    assert A.call_rope(F, over) == F.ERR_ARG


@pytest.mark.parametrize("over", [
    # an error behind that check shows that it lets these through
    dict(qots=128, qohs=5 * 128), dict(qots=-1024, qohs=128), dict(qots=1024, qohs=-128),
    dict(T=1, qots=0), dict(H=1, qohs=0), dict(kots=1024, kohs=136), dict(qots=136, qohs=8 * 136),
    dict(Hk=1, kohs=0, kots=128)], ids=str)
def test_rope_outputs_whose_rows_do_not_overlap_are_not(F, over):
    assert A.call_rope(F, dict(over, pos=A.A[4] + 4)) == F.ERR_ALIGN


@pytest.mark.parametrize("over", [
    dict(out=A.A[0]), dict(out=A.A[1]), dict(out=A.A[2]), dict(out=A.A[0], H=2, qts=256)], ids=str)
def test_prompt_output_in_place_of_an_input_is_refused(F, over):
    """Other work of the call reads rows after they are written."""
    assert A.call_prompt(F, dict(over, qs=A.A[3] + 2)) == F.ERR_ARG
