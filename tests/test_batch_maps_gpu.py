"""GPU tests of batch_extend and pages_release against a plain loop: whole numbers,
equal in every entry."""
import random

import pytest
import torch

from tests import step_ref as R
from tests.gpu_util import F

pytestmark = pytest.mark.gpu
FULL = 0x10
TOKENS = ("slot_mapping", "positions", "seq_ids", "row_lens")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(lens, width, spare, seed, capacity=None):
    """(table, free, count) as lists: random pages, -7 where the table holds none."""
    r = random.Random(seed)
    order = list(range(sum(R.pages(max(n, 0)) for n in lens) + spare))
    r.shuffle(order)
    table = []
    for n in lens:
        row = [order.pop() for _ in range(R.pages(max(n, 0)))]
        table.append(row + [-7] * (width - len(row)))
    free = order + [-9] * ((capacity or len(order)) - len(order))
    return table, free, len(order)


def run_extend(cached, new, table, free, count, T, err=True, **kw):
    d = [i32(x).reshape(s) for x, s in ((table, (len(cached), -1 if cached else 3)), (free, (-1,)),
                                        ([count], (1,)))]
    flags = i32([0])
    maps = F().batch_extend(i32(cached), i32(new), *d, T, err_flags=flags if err else None, **kw)
    torch.cuda.synchronize()
    return maps, d, int(flags)


def check_extend(cached, new, table, free, count, T, **kw):
    maps, d, flags = run_extend(cached, new, table, free, count, T, **kw)
    want, wtable, wcount, full = R.extend(cached, new, table, free, count, T)
    for name, got in maps._asdict().items():
        assert got.tolist() == want[name], name
    assert d[0].tolist() == wtable
    assert d[1].tolist() == free and int(d[2]) == wcount
    assert flags == (FULL if full else 0)
    return maps, d


@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([65], [0]), ([0], [0]), ([0], [64]), ([1], [200]),
    ([10, 64, 0, 127], [4, 4, 4, 4]), ([100, 5, 700], [0, 0, 0]), ([0, 0, 0], [130, 0, 1]),
    ([-5, 3], [2, -9])])
@pytest.mark.parametrize("slack", [0, 1, 7])
def test_small(cached, new, slack):
    table, free, count = pool(cached, 14, 20, 1)
    check_extend(cached, new, table, free, count, sum(max(n, 0) for n in new) + slack)


@pytest.mark.parametrize("B,tokens,context,seed", [
    (300, 5, 500, 1), (1025, 1, 90, 2), (4096, 2, 70, 3), (4097, 1, 200, 4), (9001, 1, 64, 5),
    (3, 20000, 3, 6), (40, 900, 1000, 7), (260, 40, 130, 8)])
def test_batches(B, tokens, context, seed):
    """Several CTAs, several thousand sequences, sequences of no new tokens."""
    r = random.Random(seed)
    cached = [r.randint(0, context) for _ in range(B)]
    new = [r.choice([0, 1, tokens, r.randint(0, tokens)]) for _ in range(B)]
    width = max(R.pages(c + n) for c, n in zip(cached, new)) + 1
    table, free, count = pool(cached, width, sum(R.pages(c + n) for c, n in zip(cached, new)), seed)
    check_extend(cached, new, table, free, count, sum(new) + seed)


@pytest.mark.parametrize("count", [0, 1, 2, 3, 5, 6, 7])
def test_too_few_free_pages(count):
    """Sequences are served in order while pages last, and after that those that
    need none."""
    cached, new = [0, 10, 64, 100, 30], [65, 5, 64, 100, 1]  # 2, 0, 1, 2 pages and none
    table, free, _ = pool(cached, 6, 7, 2)
    check_extend(cached, new, table, free, count, sum(new))


def test_a_row_that_is_too_short_and_tokens_that_do_not_fit():
    cached, new = [100, 0, 64, 3, 5], [100, 130, 64, 10, 0]
    table, free, count = pool(cached, 3, 12, 3)
    check_extend(cached, new, table, free, count, sum(new))  # the first needs 4 pages
    for T in (0, 1, 99, 100, 150, 229, 230, 294, 303, 304):
        check_extend(cached, new, table, free, count, T)


def test_the_count_is_taken_within_the_stack():
    cached, new = [0, 0], [64, 64]
    table, free, _ = pool(cached, 2, 3, 4)
    check_extend(cached, new, table, free, 99, 128)
    check_extend(cached, new, table, free, -4, 128)


def test_lengths_far_out_of_range():
    big = 2 ** 31 - 1
    for cached, new in (([big, 3], [big, 1]), ([0, 0, 0], [big, big, 5]), ([big], [0]),
                        ([5, 9], [1, big])):
        lens = [0 if c == big else c for c in cached]
        table, free, count = pool(lens, 4, 5, 5)
        maps, d, flags = run_extend(cached, new, table, free, count, 10)
        assert flags == FULL
        want = [min(sum(new[:b]), 10) for b in range(len(new) + 1)]
        assert maps.q_starts.tolist() == want
        assert maps.context_lens.tolist()[0] == (6 if cached == [5, 9] else cached[0])


def test_an_empty_pool_and_rows_without_pages():
    maps, d, flags = run_extend([5, 60], [3, 4], [[1], [2]], [], 0, 9)
    assert maps.slot_mapping.tolist() == [69, 70, 71, 188, 189, 190, 191, -1, -1] and flags == 0
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    maps = F().batch_extend(i32([0, 0]), i32([0, 1]), table, i32([]), i32([0]), 2)
    assert maps.slot_mapping.tolist() == [-1, -1] and maps.context_lens.tolist() == [0, 0]
    F().pages_release(i32([0, 100]), i32([0, 0]), table, i32([]), i32([0]))


def test_no_sequences_and_no_tokens():
    maps, d, flags = run_extend([], [], [], [3, 4], 2, 5)
    assert maps.q_starts.tolist() == [0] and maps.slot_mapping.tolist() == [-1] * 5
    assert int(d[2]) == 2 and flags == 0
    table, free, count = pool([7], 2, 2, 1)
    maps, d = check_extend([7], [0], table, free, count, 0)
    assert maps.slot_mapping.numel() == 0


def test_outputs_that_are_given_as_parts_of_wider_tensors():
    """Unaligned outputs, and a table that is part of a wider one."""
    cached, new = [100, 0, 64, 3], [30, 130, 64, 10]
    table, free, count = pool(cached, 5, 9, 3)
    T = sum(new) + 3
    wide = {n: torch.full((T + 2,), 77, dtype=torch.int64 if n in TOKENS[:2] else torch.int32,
                          device="cuda") for n in TOKENS}
    want, wtable, _, _ = R.extend(cached, new, table, free, count, T)
    big = torch.full((4, 9), 55, dtype=torch.int32, device="cuda")
    big[:, 2:7] = i32(table)
    maps = F().batch_extend(i32(cached), i32(new), big[:, 2:7], i32(free), i32([count]), T,
                            **{n: w[1:T + 1] for n, w in wide.items()})
    for n, w in wide.items():
        assert w.tolist() == [77] + want[n] + [77]
    assert big[:, 2:7].tolist() == wtable and bool((big[:, :2] == 55).all())
    assert bool((big[:, 7:] == 55).all())
    assert maps.context_lens.tolist() == want["context_lens"]


def test_each_output_may_be_missing():
    import ctypes
    f = F()
    cached, new = [100, 0, 64], [30, 130, 64]
    table, free, count = pool(cached, 4, 9, 3)
    T = sum(new)
    want, wtable, wcount, _ = R.extend(cached, new, table, free, count, T)
    names = f.BatchMaps._fields
    for left in (*names, None):  # without one, or with none at all
        c, n, t, fr, ct = i32(cached), i32(new), i32(table), i32(free), i32([count])
        outs = {m: torch.zeros(len(want[m]), device="cuda",
                               dtype=torch.int64 if m in TOKENS[:2] else torch.int32)
                for m in names if left is not None and m != left}
        p = [outs[m].data_ptr() if m in outs else None for m in names]
        st = f.lib().fp4idx_batch_extend(
            c.data_ptr(), n.data_ptr(), t.data_ptr(), 4, 4, fr.data_ptr(), ct.data_ptr(), len(free),
            *p, 3, T, None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == f.OK
        torch.cuda.synchronize()
        assert t.tolist() == wtable and int(ct) == wcount
        for m, o in outs.items():
            assert o.tolist() == want[m]


@pytest.mark.parametrize("held,kept,capacity", [
    ([200], [0], 10), ([200], [200], 10), ([200], [128], 10), ([200], [129], 10), ([0], [0], 10),
    ([64, 65, 0, 500], [0, 64, 3, 100], 30), ([64, 300], [-3, 9999], 9), ([-4, 130], [0, 1], 9),
    ([640, 640], [0, 0], 25), ([640, 640], [0, 0], 21)])
def test_release(held, kept, capacity):
    """The last two: 20 pages onto 5 in a stack of 25 and of 21 places."""
    table, free, count = pool(held, 12, 5, 7, capacity)
    d = i32(table), i32(free), i32([count])
    flags = i32([0])
    F().pages_release(i32(held), i32(kept), *d, err_flags=flags)
    want = R.release(held, kept, table, free, count)
    assert d[0].tolist() == want[0] and d[1].tolist() == want[1]
    assert int(d[2]) == want[2] and int(flags) == (FULL if want[3] else 0)


@pytest.mark.parametrize("B,context,seed", [(700, 900, 1), (1024, 64, 2), (4100, 300, 3),
                                            (9000, 130, 4), (2, 40000, 5)])
def test_release_of_large_batches(B, context, seed):
    r = random.Random(seed)
    held = [r.randint(0, context) for _ in range(B)]
    kept = [r.choice([0, h, max(h - 3, 0), r.randint(0, h)]) for h in held]
    width = max(R.pages(h) for h in held)
    table, free, count = pool(held, width, 5, seed, sum(R.pages(h) for h in held) + 5)
    d = i32(table), i32(free), i32([count])
    F().pages_release(i32(held), i32(kept), *d)
    want = R.release(held, kept, table, free, count)
    assert d[0].tolist() == want[0] and d[1].tolist() == want[1] and int(d[2]) == want[2]


def test_pages_behind_the_row_are_not_there():
    table, free, count = pool([128, 100], 2, 3, 8, 20)
    d = i32(table), i32(free), i32([count])
    F().pages_release(i32([10000, 100]), i32([64, 0]), *d)
    want = R.release([10000, 100], [64, 0], table, free, count)
    assert d[0].tolist() == want[0] and d[1].tolist() == want[1] and int(d[2]) == want[2]


def test_release_undoes_extend():
    r = random.Random(9)
    cached = [r.randint(0, 400) for _ in range(333)]
    new = [r.randint(0, 300) for _ in range(333)]
    table, free, count = pool(cached, 12, 3000, 9)
    table = [[-1 if x == -7 else x for x in row] for row in table]
    maps, d, _ = run_extend(cached, new, table, free, count, sum(new))
    F().pages_release(maps.context_lens, i32(cached), *d)
    assert d[0].tolist() == table and d[1].tolist() == free and int(d[2]) == count


def test_a_captured_step_replayed_on_its_own_lengths():
    """context_lens copied over cached_lens inside the graph: each replay goes on
    where the one before it ended."""
    cached, new = [60, 0, 127, 5], [2, 2, 2, 0]
    table, free, count = pool(cached, 8, 20, 10)
    c, n, t, fr, ct = i32(cached), i32(new), i32(table), i32(free), i32([count])
    F().batch_extend(c, n, t, fr, ct.clone(), 8)  # loads the kernel
    torch.cuda.synchronize()
    t.copy_(i32(table))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        maps = F().batch_extend(c, n, t, fr, ct, 8)
        c.copy_(maps.context_lens)
    for _ in range(70):
        want, table, count, _ = R.extend(cached, new, table, free, count, 8)
        graph.replay()
        torch.cuda.synchronize()
        for name, got in maps._asdict().items():
            assert got.tolist() == want[name], name
        assert t.tolist() == table and int(ct) == count
        cached = want["context_lens"]
    assert cached == [200, 140, 267, 5]


def test_another_stream():
    cached, new = [100, 0, 64], [30, 130, 64]
    table, free, count = pool(cached, 4, 9, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    check_extend(cached, new, table, free, count, 230, stream=side)
