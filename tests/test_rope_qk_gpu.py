"""GPU tests of rope_qk: bit for bit the formula in fp32, and within its roundings
of the formula in 64 bits."""
import pytest
import torch

from tests import step_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def tables(max_pos, half):
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return a.cos().float(), a.sin().float()


def check(x, got, positions, cos, sin, sections, interleaved, neox):
    pos = positions.view(len(sections), -1)
    y32, _ = R.rope(x, pos, cos, sin, sections, interleaved, neox, torch.float32)
    assert torch.equal(got, y32.to(x.dtype))
    y, mag = R.rope(x, pos, cos, sin, sections, interleaved, neox, torch.float64)
    u = torch.finfo(x.dtype).eps / 2
    # two products and a sum in fp32, 2^-24 of the magnitudes each, then one
    # rounding to the type (or to its subnormals)
    tol = u * y.abs() + (1 + u) * 3 * 2.0 ** -24 * mag + torch.finfo(x.dtype).tiny * u
    assert bool(((got.double() - y).abs() <= tol).all())


def run(T, Hq, Hk, D, R_dim, sections, interleaved=False, neox=True, dtype=BF, seed=0, max_pos=500):
    g = gen(seed)
    q = torch.randn(T, Hq, D, generator=g, device="cuda").to(dtype)
    k = torch.randn(T, Hk, D, generator=g, device="cuda").to(dtype) if Hk else None
    cos, sin = tables(max_pos, R_dim // 2)
    positions = torch.randint(0, max_pos, (len(sections), T), generator=g, device="cuda")
    if len(sections) == 1:
        positions = positions[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = F().rope_qk(q, k, positions, cos, sin, rope_style="neox" if neox else "interleaved",
                         sections=None if len(sections) == 1 else sections,
                         interleaved_axes=interleaved, err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(q, qo, positions, cos, sin, sections, interleaved, neox)
    if Hk:
        check(k, ko, positions, cos, sin, sections, interleaved, neox)
    else:
        assert ko is None


@pytest.mark.parametrize("T", [0, 1, 2, 7, 333])
@pytest.mark.parametrize("Hq,Hk,D,R_dim", [(1, 1, 64, 64), (32, 8, 128, 128), (3, 0, 128, 64),
                                           (5, 2, 128, 112), (7, 7, 24, 16), (2, 1, 200, 80),
                                           (1, 3, 1024, 1024), (4, 1, 1000, 16), (17, 1, 16, 16)])
@pytest.mark.parametrize("neox,dtype", [(True, BF), (False, HF)])
def test_sizes(T, Hq, Hk, D, R_dim, neox, dtype):
    run(T, Hq, Hk, D, R_dim, [R_dim // 2], neox=neox, dtype=dtype, seed=T + D)


@pytest.mark.parametrize("sections", [[16, 16], [0, 32], [32, 0], [16, 8, 8], [11, 10, 11],
                                      [0, 0, 32], [1, 30, 1], [8, 8, 8, 8], [3, 0, 20, 9],
                                      [30, 1, 1], [2, 15, 15]])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("neox", [True, False])
def test_axes(sections, interleaved, neox):
    for D in (64, 96):
        run(61, 4, 2, D, 64, sections, interleaved, neox, seed=sum(sections[:1]))


@pytest.mark.parametrize("T,Hq,Hk", [(20000, 32, 8), (3001, 1, 1), (700, 64, 64)])
def test_many_tokens(T, Hq, Hk):
    run(T, Hq, Hk, 128, 128, [24, 20, 20], seed=T, max_pos=3000)


@pytest.mark.parametrize("neox", [True, False])
def test_in_place_and_parts_of_a_projection(neox):
    g = gen(3)
    T, Hq, Hk, D = 77, 6, 2, 64
    x = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(BF)
    cos, sin = tables(100, 16)
    pos = torch.randint(0, 100, (T,), generator=g, device="cuda")
    before = x.clone()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    style = "neox" if neox else "interleaved"
    a, b = F().rope_qk(q, k, pos, cos, sin, rope_style=style)
    assert torch.equal(x, before)
    qo, ko = F().rope_qk(q, k, pos, cos, sin, rope_style=style, q_out=q, k_out=k)
    assert qo is q and torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(x[:, Hq + Hk:], before[:, Hq + Hk:])
    check(before[:, :Hq], a, pos, cos, sin, [16], False, neox)
    # queries in place, keys not, with a tail that is copied
    x.copy_(before)
    _, b2 = F().rope_qk(q, k, pos, cos, sin, rope_style=style, q_out=q)
    assert torch.equal(q, a) and torch.equal(b2, b)


def test_heads_before_tokens_and_outputs_with_strides_of_their_own():
    g = gen(4)
    T, H, D = 50, 5, 128
    q = torch.randn(H, T, D, generator=g, device="cuda").to(HF).transpose(0, 1)
    k = torch.randn(T, H, D + 8, generator=g, device="cuda").to(HF)[..., 8:]
    cos, sin = tables(64, 64)
    pos = torch.randint(0, 64, (T,), generator=g, device="cuda")
    wide = torch.full((T, 3 * H, D), 7.0, dtype=HF, device="cuda")
    out = wide[:, H:2 * H]
    F().rope_qk(q, k, pos, cos, sin, q_out=out)
    check(q, out, pos, cos, sin, [64], False, True)
    assert bool((wide[:, :H] == 7).all()) and bool((wide[:, 2 * H:] == 7).all())
    kt = torch.zeros(H, T, D, dtype=HF, device="cuda").transpose(0, 1)
    F().rope_qk(q, k, pos, cos, sin, k_out=kt)
    check(k, kt, pos, cos, sin, [64], False, True)


def test_positions_out_of_range():
    """A token with any axis out of range keeps its output rows, and is flagged."""
    g = gen(5)
    T, D = 40, 64
    q = torch.randn(T, 3, D, generator=g, device="cuda").to(BF)
    cos, sin = tables(20, 32)
    pos = torch.randint(0, 20, (2, T), generator=g, device="cuda")
    good = torch.ones(T, dtype=torch.bool)
    for t, a, p in ((3, 0, -1), (8, 1, 20), (9, 0, 2 ** 40), (39, 1, -2 ** 62)):
        pos[a, t] = p
        good[t] = False
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    F().rope_qk(q, None, pos, cos, sin, sections=[32, 0], q_out=out, err_flags=err)
    assert int(err) == 1 and bool((out[~good.cuda()] == 9).all())
    check(q[good.cuda()], out[good.cuda()], pos[:, good.cuda()].contiguous(), cos, sin, [32, 0],
          False, True)


def test_values_that_are_not_finite_stay_in_their_pairs():
    q = torch.ones(2, 1, 64, device="cuda", dtype=HF)
    q[0, 0, 5], q[1, 0, 40] = float("inf"), float("nan")
    cos, sin = tables(8, 16)  # pairs (i, i + 16) of the first 32
    out, _ = F().rope_qk(q, None, torch.tensor([3, 4], device="cuda"), cos, sin)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[0, 0, 5], [0, 0, 21], [1, 0, 40]]


def test_offsets_beyond_32_bits():
    T, H, D, step = 3, 2, 64, (1 << 30) + 64
    flat = torch.zeros((T - 1) * step + H * D, dtype=BF, device="cuda")
    q = flat.as_strided((T, H, D), (step, D, 1))
    q.copy_(torch.randn(T, H, D, generator=gen(6), device="cuda"))
    before = q.clone()
    cos, sin = tables(10, 32)
    pos = torch.tensor([9, 1, 5], device="cuda")
    F().rope_qk(q, None, pos, cos, sin, q_out=q)
    check(before, q.contiguous(), pos, cos, sin, [32], False, True)


def test_one_row_of_positions_for_all_axes():
    g = gen(8)
    q = torch.randn(30, 2, 64, generator=g, device="cuda").to(BF)
    cos, sin = tables(50, 32)
    pos = torch.randint(0, 50, (30,), generator=g, device="cuda")
    a, _ = F().rope_qk(q, None, pos, cos, sin)
    b, _ = F().rope_qk(q, None, pos.expand(3, 30), cos, sin, sections=torch.tensor([10, 11, 11]))
    c, none = F().rope_qk(q, q[:, :0], pos[None], cos, sin)
    assert torch.equal(a, b) and torch.equal(a, c) and none.shape == (30, 0, 64)


def test_strided_positions_and_another_stream():
    g = gen(7)
    T = 300
    q = torch.randn(T, 2, 64, generator=g, device="cuda").to(BF)
    cos, sin = tables(50, 32)
    wide = torch.randint(0, 50, (5, T + 9), generator=g, device="cuda")
    pos = wide[1:4:2, 4:T + 4]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, _ = F().rope_qk(q, None, pos, cos, sin, sections=[10, 22], stream=side)
    side.synchronize()
    check(q, out, pos.contiguous(), cos, sin, [10, 22], False, True)
