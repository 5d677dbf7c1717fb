"""GPU tests of the 8-bit cache's store and load against the 64-bit
definition: codes, scales and loaded values exactly."""
import pytest
import torch

from tests import kv_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cache_of(g, blocks, H, D, layout="apart"):
    kc, vc, ks, vs = R.make_cache(g, blocks, H, D)
    if layout == "apart":
        return kc, vc, ks, vs
    both = torch.empty(blocks, 2, H, 64, D, dtype=torch.uint8, device="cuda")
    sc = torch.empty(blocks, 2, H, device="cuda")
    both[:, 0], both[:, 1], sc[:, 0], sc[:, 1] = kc, vc, ks, vs
    return both[:, 0].view(torch.float8_e4m3fn), both[:, 1].view(torch.float8_e4m3fn), \
        sc[:, 0], sc[:, 1]


def check_store(k, v, slots, cache):
    kc, vc, ks, vs = cache
    want = [R.store(x, slots, c.contiguous(), s)
            for x, c, s in ((k, kc, ks), (v, vc, vs))]
    before = [c.clone() for c in (kc, vc)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    F().kv_store_fp8(k, v, slots, *cache, err_flags=err)
    torch.cuda.synchronize()
    for c, s, (val, sc), old in ((kc, ks, want[0], before[0]), (vc, vs, want[1], before[1])):
        assert torch.equal(s.double(), sc)
        got = R.codes_value(c.contiguous())
        same = (got == val) | (got.isnan() & val.isnan())
        assert bool(same.all()), int((~same).sum())
    return int(err.item())


def pattern(name, g, blocks):
    """Slots of a call."""
    dev = "cuda"
    if name == "one":
        return torch.tensor([5 * 64 + 17], device=dev)
    if name == "decode":  # a token each, on pages of their own, some skipped
        page = torch.randperm(blocks, generator=g, device=dev)
        s = page * 64 + torch.randint(0, 64, (blocks,), generator=g, device=dev)
        s[::7] = -1
        return s
    if name == "mtp":  # 5 tokens each, crossing page ends
        page = torch.randperm(blocks // 2, generator=g, device=dev)[:blocks // 4] * 2
        off = torch.randint(55, 64, (len(page),), generator=g, device=dev)
        return ((page * 64 + off)[:, None] + torch.arange(5, device=dev)).reshape(-1)
    if name == "prompts":  # ragged prompts from any offset
        parts, at = [], 0
        for n, off in ((1, 0), (64, 0), (63, 1), (65, 63), (200, 17), (9, 50), (8, 60), (130, 0)):
            parts.append(torch.arange(n, device=dev) + at * 64 + off)
            parts.append(torch.full((n % 3,), -1, dtype=torch.int64, device=dev))
            at += (off + n + 63) // 64
        assert at <= blocks
        return torch.cat(parts)
    if name == "scattered":  # pages in any order, whole and in part
        order = torch.randperm(blocks, generator=g, device=dev)[:12]
        return torch.cat([order[i] * 64 + torch.arange(64 - 5 * i, device=dev) for i in range(12)])
    raise KeyError(name)


@pytest.mark.parametrize("name", ["one", "decode", "mtp", "prompts", "scattered"])
@pytest.mark.parametrize("H,D,dtype,layout", [(1, 128, torch.bfloat16, "apart"),
                                              (3, 64, torch.float16, "halves"),
                                              (8, 128, torch.float16, "halves"),
                                              (2, 64, torch.bfloat16, "apart")])
def test_store(name, H, D, dtype, layout):
    g = gen(7)
    blocks = 40
    cache = cache_of(g, blocks, H, D, layout)
    slots = pattern(name, g, blocks).to(torch.int64).contiguous()
    T = len(slots)
    mag = torch.exp2(torch.randn(T, H, 1, generator=g, device="cuda") * 2)
    k = (torch.randn(T, H, D, generator=g, device="cuda") * mag).to(dtype)
    v = (torch.randn(T, H, D, generator=g, device="cuda") / mag).to(dtype)
    assert check_store(k, v, slots, cache) == 0


def test_store_many_tokens_uses_the_long_chunks():
    """Above 32,768 (token, head) rows a block takes 64 tokens: runs that
    cross chunks, and a call of single-token runs."""
    g = gen(11)
    H, D, blocks = 8, 128, 4200
    cache = cache_of(g, blocks, H, D)
    page = torch.randperm(blocks, generator=g, device="cuda")
    long = (page[:80, None] * 64 + torch.arange(64, device="cuda")).reshape(-1)[13:]
    single = page[80:] * 64 + torch.randint(0, 64, (blocks - 80,), generator=g, device="cuda")
    slots = torch.cat([long[:3000], single, long[3000:]])
    T = len(slots)
    assert T * H >= 64 * 512
    k = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    assert check_store(k, v, slots, cache) == 0


def test_store_strided_inputs():
    """k and v as views of a packed qkv projection."""
    g = gen(3)
    cache = cache_of(g, 8, 2, 128)
    qkv = torch.randn(100, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(100, device="cuda") + 64 + 5
    assert check_store(qkv[:, 4:6], qkv[:, 6:8], slots, cache) == 0


def test_store_grows_and_never_shrinks_a_scale():
    g = gen(5)
    cache = cache_of(g, 4, 1, 128)
    one = torch.ones(1, 1, 128, device="cuda", dtype=torch.bfloat16)
    slot = torch.tensor([64], device="cuda")
    for i, mag in enumerate((1.0, 3.0, 448.0, 0.01, 1e30, 1e-30, 449.0, 0.0)):
        assert check_store(one * mag, one * -mag, slot + i, cache) == 0
    # offset 0 starts anew
    assert check_store(one * 0.0, one * 1e-38, slot, cache) == 0
    assert float(cache[2][1, 0]) == 2.0 ** -126


def test_store_skips_out_of_range_slots_and_their_values():
    g = gen(9)
    cache = cache_of(g, 4, 2, 64)
    slots = torch.tensor([3, 4, -1, 5, 4 * 64, 6, 2 ** 40, -2 ** 62], device="cuda")
    k = torch.randn(8, 2, 64, generator=g, device="cuda").to(torch.float16)
    v = torch.randn(8, 2, 64, generator=g, device="cuda").to(torch.float16)
    for i in (2, 4, 6, 7):
        k[i], v[i] = float("nan"), float("inf")
    # 3, 4 | 5 | 6 are three runs of one page: only the scales and rows of the
    # last of them are fixed by the definition, so give each its own page
    slots = torch.tensor([3, 4, -1, 64 + 5, 4 * 64, 128 + 6, 2 ** 40, -2 ** 62], device="cuda")
    assert check_store(k, v, slots, cache) == F_SLOT


F_SLOT = 0x2


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("T", [1, 7, 64, 1001])
def test_load(T, D, dtype):
    g = gen(T)
    H, blocks = 3, 9
    kc, vc, ks, vs = cache_of(g, blocks, H, D, "halves" if T % 2 else "apart")
    ks.mul_(2.0 ** -100)
    slots = torch.randint(-30, blocks * 64 + 20, (T,), generator=g, device="cuda")
    k0 = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    v0 = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    ko, vo = k0.clone(), v0.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    F().kv_load_fp8(kc, vc, ks, vs, slots, k_out=ko, v_out=vo, err_flags=err)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < blocks * 64)
    at = slots[live]
    for got, old, c, s in ((ko, k0, kc, ks), (vo, v0, vc, vs)):
        val = R.codes_value(c.contiguous())[at // 64, :, at % 64] * s[at // 64].double()[..., None]
        assert torch.equal(got[live], val.float().to(dtype))  # exact, or one rounding
        assert torch.equal(got[~live], old[~live])
    assert int(err.item()) == (F_SLOT if bool((slots >= blocks * 64).any()) else 0)


def test_store_then_load_round_trip():
    """What was stored comes back within half a code step of its value."""
    g = gen(1)
    cache = cache_of(g, 8, 2, 128)
    k = torch.randn(300, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(300, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(300, device="cuda") + 64
    F().kv_store_fp8(k, v, slots, *cache)
    ko, vo = F().kv_load_fp8(*cache, slots)
    for x, y, s in ((k, ko, cache[2]), (v, vo, cache[3])):
        scale = s[slots // 64].double()[..., None]
        tol = x.double().abs() * 2.0 ** -4 + scale * 2.0 ** -10
        assert bool(((y.double() - x.double()).abs() <= tol).all())


def test_empty_calls():
    g = gen(2)
    cache = cache_of(g, 2, 1, 64)
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    F().kv_store_fp8(none, none, slots, *cache)
    ko, vo = F().kv_load_fp8(*cache, slots)
    assert ko.shape == (0, 1, 64) and vo.shape == (0, 1, 64)


def test_offsets_past_32_bits():
    """Pages whose code offsets pass 2^32 bytes."""
    H, D, blocks = 8, 128, 70000  # 65,536 bytes a block and side, halves of one tensor
    both = torch.empty(blocks, 2, H, 64, D, dtype=torch.uint8, device="cuda")
    sc = torch.ones(blocks, 2, H, device="cuda")
    cache = (both[:, 0], both[:, 1], sc[:, 0], sc[:, 1])
    g = gen(4)
    T = 70
    k = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(T, device="cuda") + (blocks - 2) * 64
    F().kv_store_fp8(k, v, slots, *cache)
    small = [c[-2:].contiguous() for c in cache]
    fresh = [torch.zeros_like(c) for c in small]
    F().kv_store_fp8(k, v, slots - (blocks - 2) * 64, *fresh)
    torch.cuda.synchronize()
    assert torch.equal(small[2], fresh[2]) and torch.equal(small[3], fresh[3])
    for a, b in zip(small[:2], fresh[:2]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1, :, :T - 64], b[1, :, :T - 64])
    ko, vo = F().kv_load_fp8(*cache, slots)
    kf, vf = F().kv_load_fp8(*fresh, slots - (blocks - 2) * 64)
    assert torch.equal(ko, kf) and torch.equal(vo, vf)
    # attention over them
    q = torch.randn(1, 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    far = torch.tensor([[blocks - 2, blocks - 1]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([T], dtype=torch.int32, device="cuda")
    a = F().paged_attention_fp8(q, *cache, far, ctx, 128)
    b = F().paged_attention_fp8(q, *fresh, near, ctx, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
