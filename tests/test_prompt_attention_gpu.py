"""GPU tests of prompt_attention against the 64-bit definition within derived
bounds (step_ref.check)."""
import pytest
import torch

from tests import step_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prefix(x):
    got = [0]
    for n in x:
        got.append(got[-1] + n)
    return got


def inputs(qs, ks, H, Hk, D, dtype, seed, spread=1.5):
    g = gen(seed)
    q = (torch.randn(sum(qs), H, D, generator=g, device="cuda") * spread).to(dtype)
    k, v = (torch.randn(sum(ks), Hk, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    return q, k, v


def call(q, k, v, qs, ks, whole, window=0, sinks=0, scale=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if not whole:
        kw.update(k_starts=i32(prefix(ks)), max_k=max(ks) if ks else 0)
    kw.setdefault("max_q", max(max(qs), 1))
    out, lse = F().prompt_attention(q, k, v, i32(prefix(qs)), window=window, sinks=sinks,
                                    softmax_scale=scale, err_flags=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out, lse


def run(qs, H, Hk, D, dtype, ks=None, window=0, sinks=0, seed=0, spread=1.5, scale=None):
    q, k, v = inputs(qs, ks or qs, H, Hk, D, dtype, seed, spread)
    out, lse = call(q, k, v, qs, ks or qs, ks is None, window, sinks, scale)
    ref = R.attend(q, k, v, prefix(qs), prefix(ks or qs), window, sinks,
                   D ** -0.5 if scale is None else scale)
    R.check(out, lse, ref)
    return out, lse


HEADS = [(8, 1, 128, BF), (6, 2, 64, HF), (5, 5, 128, HF), (14, 2, 128, BF), (3, 1, 64, BF)]


@pytest.mark.parametrize("qs", [[1], [2], [63], [64], [127], [128], [129], [255], [256], [257],
                                [1, 1, 1], [0, 5, 0], [300, 0, 1, 64, 129, 3]])
@pytest.mark.parametrize("H,Hk,D,dtype", HEADS)
def test_whole_prompts(qs, H, Hk, D, dtype):
    run(qs, H, Hk, D, dtype, seed=sum(qs) + H)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 70), (128, 0), (129, 130),
                                          (500, 3), (5000, 3)])
@pytest.mark.parametrize("H,Hk,D,dtype", [(4, 1, 128, BF), (7, 1, 64, HF), (2, 2, 64, BF)])
def test_windows(window, sinks, H, Hk, D, dtype):
    run([700, 1, 130], H, Hk, D, dtype, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("qs,ks", [([1], [1]), ([1], [1000]), ([4], [129]), ([40, 1], [300, 2000]),
                                   ([1, 1, 1, 1], [64, 0, 1, 513]), ([200, 3], [100, 0]),
                                   ([130, 64], [1, 640]), ([33], [4000]), ([300, 5], [5, 300])])
@pytest.mark.parametrize("H,Hk,D,dtype,window,sinks", [
    (8, 1, 128, BF, 0, 0), (6, 2, 64, HF, 0, 0), (5, 1, 128, HF, 130, 0), (8, 2, 64, BF, 50, 200),
    (130, 1, 128, BF, 0, 0), (260, 2, 64, BF, 300, 4)])
def test_queries_at_the_end_of_longer_or_shorter_keys(qs, ks, H, Hk, D, dtype, window, sinks):
    """Chunks and single tokens; fewer keys than queries leave the first rows
    without one."""
    run(qs, H, Hk, D, dtype, ks, window, sinks, seed=sum(ks) + H)


@pytest.mark.parametrize("qs,H,Hk,D,dtype,window", [
    ([5000], 2, 1, 128, BF, 0), ([3000, 17, 1024], 4, 2, 64, HF, 0), ([2500, 900], 12, 4, 128, HF, 0),
    ([4000, 4000], 1, 1, 64, BF, 600), ([37] * 70, 4, 4, 128, BF, 0), ([700] * 9, 6, 2, 64, HF, 0)])
def test_long_and_many(qs, H, Hk, D, dtype, window):
    """Items of many tiles, cut between CTAs and joined; more items than CTAs."""
    run(qs, H, Hk, D, dtype, window=window, seed=len(qs))


@pytest.mark.parametrize("G,Hk", [(16, 2), (32, 1), (64, 2), (128, 1), (24, 1), (100, 1)])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, HF)])
def test_large_groups(G, Hk, D, dtype):
    """Up to 128 heads over one: a warp's rows, a half and an item are a few tokens or
    part of one."""
    run([70, 3, 1], G * Hk, Hk, D, dtype, seed=G)
    run([5, 1], G * Hk, Hk, D, dtype, ks=[400, 2], window=90, sinks=3, seed=G)


def test_thousands_of_sequences():
    import random
    r = random.Random(2)
    qs = [r.choice([0, 1, 1, 2, 3, 40]) for _ in range(3000)]
    run(qs, 4, 2, 64, BF, seed=1)
    ks = [n + r.randint(0, 30) for n in qs]
    run(qs, 4, 2, 64, BF, ks=ks, seed=2)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_along_the_keys(dtype, D, rising):
    """The reference of the sums moves in every tile, or never after the first."""
    n, H = 900, 2
    g = gen(3)
    d = torch.randn(D, generator=g, device="cuda")
    d /= d.norm()
    ramp = torch.linspace(-30, 30, n, device="cuda") * (1 if rising else -1)
    k = (ramp[:, None] * d + 0.3 * torch.randn(n, D, generator=g, device="cuda"))[:, None].to(dtype)
    q = (6 * d + 0.2 * torch.randn(n, H, D, generator=g, device="cuda")).to(dtype)
    v = torch.randn(n, 1, D, generator=g, device="cuda").to(dtype)
    out, lse = call(q, k, v, [n], [n], True, scale=1.0)
    R.check(out, lse, R.attend(q, k, v, [0, n], [0, n], 0, 0, 1.0))


@pytest.mark.parametrize("scale", [0.0, 1e-30, 3.0])
def test_scales(scale):
    run([150, 2], 4, 2, 64, BF, seed=5, scale=scale, spread=0.5)


def test_rows_in_no_sequence_may_hold_anything_and_stay():
    """A padded batch: NaN in the rows behind the last sequence, and between two, of
    q, k and v; nothing of out and lse is written there."""
    qs, H, Hk, D = [130, 70], 4, 2, 128
    g = gen(6)
    T = 300
    q = torch.randn(T, H, D, generator=g, device="cuda").to(BF)
    k, v = (torch.randn(T, Hk, D, generator=g, device="cuda").to(BF) for _ in range(2))
    # the first ends at 130, the second one's rows are 130 .. 199
    for t in (q, k, v):
        t[200:] = NAN
    out = torch.full((T, H, D), 3.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 3.0, device="cuda")
    call(q, k, v, qs, qs, True, out=out, lse=lse)
    assert bool((out[200:] == 3).all()) and bool((lse[200:] == 3).all())
    R.check(out[:200], lse[:200], R.attend(q[:200], k[:200], v[:200], [0, 130, 200],
                                           [0, 130, 200], 0, 0, D ** -0.5))
    # sequences that do not begin at 0
    out.fill_(3.0)
    starts = i32([10, 60, 60, 200])
    F().prompt_attention(q, k, v, starts, 140, out=out, lse=lse)
    assert bool((out[:10] == 3).all()) and bool((out[200:] == 3).all())
    ref = R.attend(q, k, v, [10, 60, 60, 200], [10, 60, 60, 200], 0, 0, D ** -0.5)
    R.check(out[10:200], lse[10:200], tuple(x[10:200] for x in ref))


def test_what_one_sequence_holds_reaches_no_other():
    """Infinities and NaN in one sequence's keys, values and queries; its neighbours
    share its tiles of 128 keys."""
    qs, H, Hk, D = [50, 60, 40, 200], 6, 2, 64
    q, k, v = inputs(qs, qs, H, Hk, D, HF, 7)
    want = call(q, k, v, qs, qs, True)
    for bad in (NAN, float("inf"), -float("inf")):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[50:110] = bad
        for window in (0, 30):
            want = call(q, k, v, qs, qs, True, window=window)
            out, lse = call(q2, k2, v2, qs, qs, True, window=window)
            for rows in (slice(0, 50), slice(110, 350)):
                assert torch.equal(out[rows], want[0][rows])
                assert torch.equal(lse[rows], want[1][rows])


def test_keys_that_no_query_sees_may_hold_anything():
    """Below the window and behind the first tokens, and behind max_k."""
    qs, ks, D = [5], [1000], 128
    q, k, v = inputs(qs, ks, 8, 2, D, BF, 8)
    want = call(q, k, v, qs, ks, False, window=100, sinks=7)
    for t in (k, v):
        t[7:1000 - 104] = NAN
    got = call(q, k, v, qs, ks, False, window=100, sinks=7)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # keys behind the 500th are not seen
    q, k, v = inputs([600], [600], 4, 1, D, BF, 9)
    v[500:] = NAN
    out, lse = F().prompt_attention(q, k, v, i32([0, 600]), 600, max_k=500)
    ref = R.attend(q, k, torch.nan_to_num(v), [0, 600], [0, 600], 0, 0, D ** -0.5, max_k=500)
    R.check(out, lse, ref)


@pytest.mark.parametrize("n,before", [(200, 0), (1, 5000)])
def test_a_row_with_a_nan_is_nan_and_no_other(n, before):
    """Also where the row's keys are shared out among CTAs."""
    q, k, v = inputs([n], [n + before], 2, 1, 64, HF, 10)
    want = call(q, k, v, [n], [n + before], False)
    q2 = q.clone()
    q2[n // 3, 1, 3] = NAN
    out, lse = call(q2, k, v, [n], [n + before], False)
    assert bool(torch.isnan(out[n // 3, 1]).all()) and bool(torch.isnan(lse[n // 3, 1]))
    keep = torch.ones(n, 2, dtype=torch.bool, device="cuda")
    keep[n // 3, 1] = False
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_tokens_behind_max_q_are_left_unwritten():
    q, k, v = inputs([400], [400], 4, 2, 64, BF, 11)
    ref = R.attend(q, k, v, [0, 400], [0, 400], 0, 0, 64 ** -0.5)
    for max_q in (1, 100, 399):
        out = torch.full_like(q, 3.0)
        lse = torch.full((400, 4), 3.0, device="cuda")
        F().prompt_attention(q, k, v, i32([0, 400]), max_q, max_k=400, out=out, lse=lse)
        R.check(out[:max_q], lse[:max_q], tuple(x[:max_q] for x in ref))
        assert bool((out[max_q:] == 3).all()) and bool((lse[max_q:] == 3).all())


@pytest.mark.parametrize("max_k", [1, 100, 128, 300, 599])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3), (100, 0), (300, 40), (400, 0), (600, 0)])
def test_keys_behind_max_k_are_not_seen(max_k, window, sinks):
    """A window ends at the query, which may stand behind the last key that counts."""
    qs, ks = [130, 2], [600, 90]
    q, k, v = inputs(qs, ks, 4, 2, 64, BF, max_k + window)
    ref = R.attend(q, k, v, prefix(qs), prefix(ks), window, sinks, 64 ** -0.5, max_k=max_k)
    out, lse = F().prompt_attention(q, k, v, i32(prefix(qs)), 130, k_starts=i32(prefix(ks)),
                                    max_k=max_k, window=window, sinks=sinks)
    R.check(out, lse, ref)


@pytest.mark.parametrize("D,dtype", [(128, BF), (64, HF)])
@pytest.mark.parametrize("H,Hk", [(8, 2), (6, 2), (3, 3)])
def test_layouts(D, dtype, H, Hk):
    """Parts of one projection, heads before tokens, padded rows, one key tensor for
    all heads, keys as values, single heads of wider tensors."""
    n = 333
    g = gen(12)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    x = rand(n, H + 2 * Hk, D)
    heads_first = rand(H, n, D).transpose(0, 1)
    kv = rand(Hk, n + 11, D)[:, 5:n + 5].transpose(0, 1)
    wide = rand(n, Hk, D + 24)[..., 16:16 + D]
    q0, k0, v0 = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    cases = [(q0, k0, v0), (heads_first, kv, v0), (q0, wide, kv), (q0, k0, k0),
             (q0, k0[:, :1].expand(n, Hk, D), v0), (rand(n, H, D + 8)[..., :D], k0, wide),
             (q0, rand(n, 2 * Hk, D)[:, ::2], v0), (rand(n, 2 * H, D)[:, ::2], k0, v0),
             (rand(2 * n, H, D)[::2], rand(3 * n, Hk, D)[::3], v0)]
    if Hk > 1:
        cases.append((q0, rand(Hk, n, D).transpose(0, 1), rand(Hk, n, D).transpose(0, 1)))
    for q, k, v in cases:
        out, lse = call(q, k, v, [n - 40, 40], [n - 40, 40], True)
        R.check(out, lse, R.attend(q, k, v, [0, n - 40, n], [0, n - 40, n], 0, 0, D ** -0.5))


def test_offsets_beyond_32_bits():
    n, D, step = 150, 64, (1 << 24) + 128
    flat = torch.zeros((n - 1) * step + 2 * D, dtype=BF, device="cuda")
    x = flat.as_strided((n, 2, D), (step, D, 1))
    x.copy_(torch.randn(n, 2, D, generator=gen(13), device="cuda"))
    out, lse = call(x, x, x, [n], [n], True)
    R.check(out, lse, R.attend(x, x, x, [0, n], [0, n], 0, 0, D ** -0.5))


def test_no_keys_at_all():
    q = torch.randn(5, 4, 64, device="cuda").to(BF)
    kv = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    out, lse = F().prompt_attention(q, kv, kv, i32([0, 2, 5]), 3, k_starts=i32([0, 0, 0]), max_k=0)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    out, lse = F().prompt_attention(q[:0], kv, kv, i32([0]), 1)
    assert out.shape == (0, 4, 64)
    out = torch.full_like(q, 2.0)
    F().prompt_attention(q, q[:, :2], q[:, :2], i32([0, 0]), 1, out=out)  # a batch of nothing
    assert bool((out == 2).all())


def test_starts_out_of_order_or_range_stay_within_the_tensors():
    q, k, v = inputs([100], [100], 4, 2, 64, BF, 14)
    for starts in ([-5, 100], [0, 10 ** 9], [90, 20, 100], [2 ** 31 - 1, -2 ** 31, 7]):
        out, lse = F().prompt_attention(q, k, v, i32(starts), 100, max_k=100)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).any())


def test_calls_repeat_themselves_whatever_the_workspace_holds():
    qs, ks = [1, 40, 700], [3000, 2000, 700]
    q, k, v = inputs(qs, ks, 8, 2, 128, BF, 15)
    n = F().prompt_workspace_bytes(3, 700, 8, 2, 128)
    want = None
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        got = call(q, k, v, qs, ks, False, workspace=ws)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_on_two_streams():
    qs, ks = [300, 2, 900], [300, 1200, 1000]
    q, k, v = inputs(qs, ks, 8, 2, 128, BF, 16)
    q64, k64, v64 = inputs([500, 500], [500, 500], 6, 2, 64, HF, 17)
    st, kst, st64 = i32(prefix(qs)), i32(prefix(ks)), i32([0, 500, 1000])

    def one():
        return F().prompt_attention(q, k, v, st, 900, k_starts=kst, max_k=1200)

    def two():
        return F().prompt_attention(q64, k64, v64, st64, 500, window=200, sinks=2)

    want = one(), two()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one(), two()
    for scale in (1, 2):
        q.mul_(scale)
        want = one(), two()
        for a in (*got[0], *got[1]):
            a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got[0], *got[1]), (*want[0], *want[1])):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(8):
        for s, fn in zip(streams, (one, two)):
            with torch.cuda.stream(s):
                outs.append(fn())
    torch.cuda.synchronize()
    for i, pair in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(pair, want[i % 2]))


def test_many_passes_of_ragged_batches():
    """Items with and without a second half in every order: no wait runs out, and
    every pass gives the first one's bits."""
    import random
    r = random.Random(5)
    for D, G in ((64, 1), (128, 4), (64, 7), (128, 1)):
        qs = [r.choice([1, 5, 31, 130, 256, 300, 900]) for _ in range(40)]
        q, k, v = inputs(qs, qs, 2 * G, 2, D, BF, D + G)
        st = i32(prefix(qs))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        first = None
        for i in range(150):
            got = F().prompt_attention(q, k, v, st, 900, window=200 if i % 2 else 0, err_flags=err)
            if i < 2:
                first = (*(first or ()), [t.clone() for t in got])
            elif i % 7 == 0:
                assert all(torch.equal(a, b) for a, b in zip(got, first[i % 2]))
        torch.cuda.synchronize()
        assert int(err) == 0


@pytest.mark.parametrize("index", [0, 3])
def test_a_wait_that_runs_out(index):
    """The keys of a tile of CTA 0 are withheld: the launch returns after a second
    with the flag alone, other CTAs' rows are right, the next launch is."""
    f = F()
    q, k, v = inputs([2000] * 4, [2000] * 4, 8, 8, 128, BF, 18)
    st = i32(prefix([2000] * 4))
    want = f.prompt_attention(q, k, v, st, 2000)
    torch.cuda.synchronize()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    f.test_withhold_next(f.TEST_PROMPT, index)
    out, lse = f.prompt_attention(q, k, v, st, 2000, err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == f.ERRFLAG_TIMEOUT
    # the last sequence is other CTAs' work
    assert torch.equal(out[7000:], want[0][7000:]) and torch.equal(lse[7000:], want[1][7000:])
    err.zero_()
    out, lse = f.prompt_attention(q, k, v, st, 2000, err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_an_index_behind_the_work_withholds_nothing():
    f = F()
    q, k, v = inputs([50], [50], 4, 2, 64, BF, 19)
    for index in (1000, 1 << 40):
        f.test_withhold_next(f.TEST_PROMPT, index)
        call(q, k, v, [50], [50], True)
