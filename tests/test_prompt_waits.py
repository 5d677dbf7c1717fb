"""The barriers of attention of prompts, as a model on the CPU.

A wait on a barrier's phase is a test of its parity, so it is sound only if the
barrier cannot complete a second phase before the waiting warp has looked.  Roles
are straight programs of waits and arrivals and barriers only count, so the
furthest that the others can get while one role stands still before a wait is
found by running them until none moves."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "fp4_sparse_attention_fp4idx_gb300", "csrc", "fp4idx_prompt.cu")


def source():
    """Ring sizes by head size, the clean ring, the segment ring and whether warps
    2 and 3 wait for key tiles as well, from the kernel's text."""
    with open(SOURCE) as f:
        text = f.read()
    a, b = re.search(r"ring_of\(int D\) \{ return D == 128 \? (\d+) : (\d+); \}", text).groups()
    clean, = re.search(r"kCleanRing = (\d+);", text).groups()
    segs, = re.search(r"kSegRing = (\d+);", text).groups()
    side = text[text.index("queries, unseen value rows"):text.index("MMA issuer\n")]
    return {128: int(a), 64: int(b)}, int(clean), int(segs), side.count("wait(B::kFullAt") > 1


def arrivals(bar):
    return {"seg_empty": 11, "p_half": 4, "p_full": 4, "clean": 2}.get(bar[0], 1)


def programs(segments, ring, clean, segs, key_wait):
    """The waits and arrivals of every role for segments of (tiles, halves): a copy or
    a product is taken to be done where it is asked for."""
    def wait(*bar_and_phase):
        return ("wait", bar_and_phase[:-1], bar_and_phase[-1])

    def arrive(*bar):
        return ("arrive", bar, 0)

    roles = {}
    ops = roles["load"] = []
    u = 0
    for i, (tiles, _) in enumerate(segments):
        if i >= segs:
            ops.append(wait("seg_empty", i % segs, i // segs - 1))
        ops.append(arrive("seg_full", i % segs))
        for _ in range(2 * tiles):
            if u >= ring:
                ops.append(wait("empty", u % ring, u // ring - 1))
            ops.append(arrive("full", u % ring))
            u += 1

    def segment(ops, i):
        ops += [wait("seg_full", i % segs, i // segs), arrive("seg_empty", i % segs)]

    for half in (0, 1):
        ops = roles["side", half] = []
        n = fills = 0
        for i, (tiles, halves) in enumerate(segments):
            segment(ops, i)
            if halves > half:
                if fills:
                    ops.append(wait("q_empty", half, fills - 1))
                ops.append(arrive("q_full", half))
                fills += 1
            for _ in range(tiles):
                for u in ((2 * n, 2 * n + 1) if key_wait else (2 * n + 1,)):
                    ops.append(wait("full", u % ring, u // ring))
                ops.append(arrive("clean", n % clean))
                n += 1

    ops = roles["issue"] = []
    n, tiles_of, q_of, at = 0, [0, 0], [0, 0], 0
    for i, (tiles, halves) in enumerate(segments):
        segment(ops, i)
        ops.append(wait("full", at % ring, at // ring))
        for h in range(halves):
            ops += [wait("q_full", h, q_of[h]), arrive("s_full", h)]
            q_of[h] += 1
        at += 1
        for t in range(tiles):
            last = t + 1 == tiles
            at += 1
            ops.append(wait("clean", n % clean, n // clean))
            if not last:
                ops.append(wait("full", at % ring, at // ring))
            for h in range(halves):
                ops += [wait("p_half", h, tiles_of[h]), wait("p_full", h, tiles_of[h]),
                        arrive("o_done" if last else "s_full", h)]
                tiles_of[h] += 1
            n += 1
            at += not last

    for half in (0, 1):
        for warp in range(4):
            ops = roles["softmax", half, warp] = []
            n = every = done = 0
            for i, (tiles, halves) in enumerate(segments):
                segment(ops, i)
                if half >= halves:
                    every += tiles
                    continue
                says_all = warp == 0 and half == halves - 1
                for t in range(tiles):
                    ops.append(wait("s_full", half, n))
                    if says_all:
                        if t:
                            ops.append(arrive("empty", (2 * every - 1) % ring))
                        ops.append(arrive("empty", 2 * every % ring))
                    if warp == 0 and t + 1 == tiles:
                        ops.append(arrive("q_empty", half))
                    ops += [arrive("p_half", half), arrive("p_full", half)]
                    n += 1
                    every += 1
                ops.append(wait("o_done", half, done))
                done += 1
                if says_all:
                    ops.append(arrive("empty", (2 * every - 1) % ring))
    return roles


def run(roles, count, at, held=None):
    """Runs all roles but `held` as far as they get; counts of arrivals in `count`,
    places in the programs in `at`, both in place."""
    moved = True
    while moved:
        moved = False
        for role, ops in roles.items():
            while role != held and at[role] < len(ops):
                kind, bar, phase = ops[at[role]]
                if kind == "wait" and count.get(bar, 0) // arrivals(bar) <= phase:
                    break
                if kind == "arrive":
                    count[bar] = count.get(bar, 0) + 1
                at[role] += 1
                moved = True


def overtaken(roles):
    """The waits, as (role, barrier), whose phase and the next one can both complete
    before the role has looked."""
    found = set()
    for role, ops in roles.items():
        for place, (kind, bar, phase) in enumerate(ops):
            if kind != "wait":
                continue
            # the role as far as this wait, the others as far as they get
            count, at = {}, dict.fromkeys(roles, 0)
            run({**roles, role: ops[:place]}, count, at)
            assert at[role] == place
            if count.get(bar, 0) // arrivals(bar) > phase + 1:
                found.add((role, bar))
    return found


def segments_of(seed):
    r = random.Random(seed)
    return [(r.choice([1, 1, 2, 3, 7]), r.choice([1, 2])) for _ in range(r.choice([3, 6]))]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seed", range(8))
def test_no_phase_is_overtaken(D, seed):
    rings, clean, segs, key_wait = source()
    roles = programs(segments_of(seed), rings[D], clean, segs, key_wait)
    count, at = {}, dict.fromkeys(roles, 0)
    run(roles, count, at)
    assert at == {role: len(ops) for role, ops in roles.items()}  # all end
    assert overtaken(roles) == set()


@pytest.mark.parametrize("D", [64, 128])
def test_the_model_sees_a_wait_that_nothing_holds(D):
    """Warps 2 and 3 waiting for key tiles too: a key tile's place is given back by
    the softmax, whether or not they have looked."""
    rings, clean, segs, _ = source()
    roles = programs([(9, 2)], rings[D], clean, segs, True)
    assert {role for role, _ in overtaken(roles)} == {("side", 0), ("side", 1)}
