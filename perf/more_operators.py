"""Cases and plain forms of the operators around the caches: pages and maps of
a step built on the GPU, rotary positions of several axes on the main queries
and keys, and attention of packed prompts over their own keys in 16 bits.

Every operator has a plain form in elementary torch operations (fp32, rounded
once at the end), the call of the framework's own kernels (`own`), and, where
its outputs are computed numbers, its definition in 64 bits (`exact`).

Pages hold 64 tokens: token p of sequence b lives at page block_table[b, p // 64],
offset p % 64, slot page * 64 + offset.  Free pages are a stack, taken from the
top.  Packed sequences: tokens starts[b] .. starts[b+1] - 1 belong to sequence b.
"""
import math
import random

import torch

own = False

PAGE = 64
NEG = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few chats, four drafted tokens each, all of them rejected: pages
        # and maps for the step, then the pages taken back
        dict(name="draft_small", op="draft", batch=7, tokens=4, context=1000, slack=0),
        # the same for a large serving batch, the step padded to a fixed size
        dict(name="draft_large", op="draft", batch=3000, tokens=2, context=8000, slack=144),
        # finished requests give their pages back and new prompts take them:
        # some 60,000 tokens of a prefill step padded to a fixed size
        dict(name="turnover_prefill", op="turnover", batch=256, share=16, context=8000,
             slack=4099),
        # one decode step of nine sequences
        dict(name="rope_decode", op="rope", tokens=9, heads=32, kv_heads=8, dim=128, rotary=128,
             axes=1, order="sections", style="neox", fused=False, dtype="bf16"),
        # a packed prefill step, queries and keys as parts of one projection
        dict(name="rope_prompt", op="rope", tokens=16384, heads=32, kv_heads=8, dim=128,
             rotary=128, axes=1, order="sections", style="neox", fused=True, dtype="bf16"),
        # video frames between text: time, height, width by ranges of the pairs
        dict(name="rope_video", op="rope", tokens=30011, heads=16, kv_heads=2, dim=128,
             rotary=128, axes=3, order="sections", style="neox", fused=False, dtype="bf16"),
        # images: height and width dealt in turn, half of each head rotated
        dict(name="rope_image", op="rope", tokens=4100, heads=16, kv_heads=16, dim=64, rotary=32,
             axes=2, order="interleaved", style="interleaved", fused=False, dtype="fp16"),
        # five short chats, first tokens of a conversation
        dict(name="prompt_short", op="prompt", batch=5, q=60, context=0, heads=32, kv_heads=8,
             dim=128, window=0, sinks=0, slack=0, dtype="bf16"),
        # a packed batch of ragged prompts, padded behind the last one
        dict(name="prompt_batch", op="prompt", batch=16, q=4000, context=0, heads=32, kv_heads=8,
             dim=128, window=0, sinks=0, slack=91, dtype="bf16"),
        # one long document
        dict(name="prompt_long", op="prompt", batch=1, q=16384, context=0, heads=64, kv_heads=8,
             dim=128, window=0, sinks=0, slack=0, dtype="bf16"),
        # a sliding-window layer with four sinks, heads not grouped
        dict(name="prompt_window", op="prompt", batch=2, q=8001, context=0, heads=24, kv_heads=24,
             dim=64, window=1024, sinks=4, slack=0, dtype="fp16"),
        # single tokens of a batch over contiguous keys in 16 bits
        dict(name="prompt_single", op="prompt", batch=32, q=1, context=20000, heads=32,
             kv_heads=4, dim=128, window=0, sinks=0, slack=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["draft", "turnover", "rope", "rope", "prompt", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "draft":
        return dict(op=op, batch=_log(rng, 1, 3000), tokens=rng.choice([1, 1, 2, 4, 5]),
                    context=_log(rng, 1, 8000), slack=rng.choice([0, 0, 3, 100]))
    if op == "turnover":
        share = rng.choice([1, 3, 16])
        return dict(op=op, batch=_log(rng, 1, 16 * share), share=share,
                    context=_log(rng, 1, 8000), slack=rng.choice([0, 17, 1000]))
    if op == "rope":
        kv = rng.choice([1, 2, 5, 8])
        heads = kv * rng.choice([1, 3, 4, 8])
        dim = rng.choice([128, 128, 64])
        axes = rng.choice([1, 2, 3])
        return dict(op=op, tokens=_log(rng, 1, min(30000, 600000 // (heads + kv))), heads=heads,
                    kv_heads=kv, dim=dim, rotary=rng.choice([dim, dim, dim // 2]), axes=axes,
                    order=rng.choice(["sections", "interleaved"]),
                    style=rng.choice(["neox", "interleaved"]), fused=rng.random() < 0.5,
                    dtype=dtype)
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 3, 4, 7, 8])
    dim = rng.choice([128, 128, 64])
    window = rng.choice([0, 0, 0, 100, 1000])
    sinks = rng.choice([0, 4, 70]) if window else 0
    slack = rng.choice([0, 0, 1, 50])
    kind = rng.random()
    if kind < 0.25:  # single and drafted tokens over contiguous keys
        context = _log(rng, 1, 20000)
        batch = max(1, min(_log(rng, 1, 64), 300000 // context))
        return dict(op=op, batch=batch, q=rng.choice([1, 1, 2, 4]), context=context, heads=heads,
                    kv_heads=kv, dim=dim, window=window, sinks=sinks, slack=slack, dtype=dtype)
    q = _log(rng, 1, 8000)
    context = _log(rng, 1, 4000) if kind < 0.45 else 0  # a chunk, or whole prompts
    batch = max(1, min(_log(rng, 1, 40), 24000 // (q + context)))
    return dict(op=op, batch=batch, q=q, context=context, heads=heads, kv_heads=kv, dim=dim,
                window=window, sinks=sinks, slack=slack, dtype=dtype)


def _spread(n, top, least=1):
    """n lengths up to `top`, the first the longest, the same for every seed."""
    return [max(least, int(top * (1.0 - 0.75 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]


def _draft_lengths(case):
    """(cached, new) lengths; a sequence in the middle pauses."""
    B = case["batch"]
    new = [case["tokens"]] * B
    if B > 2:
        new[B // 2] = 0
    return _spread(B, case["context"], 0), new


def _turnover_lengths(case):
    """Lengths before and after: every `share`-th request has finished, and a
    prompt of as many pages takes its place."""
    held = _spread(case["batch"], case["context"])
    kept = [0 if i % case["share"] == 0 else n for i, n in enumerate(held)]
    new = [n - (i % 5 if (n - 1) % PAGE >= 5 else 0) if k == 0 else 0
           for i, (n, k) in enumerate(zip(held, kept))]
    return held, kept, new


def _prompt_lengths(case):
    """(query lengths, key lengths); the last query token stands at the last key."""
    qs = _spread(case["batch"], case["q"])
    before = _spread(case["batch"], case["context"]) if case["context"] else [0] * case["batch"]
    return qs, [n + c for n, c in zip(qs, before)]


def _visible(case):
    """Keys that any query of a sequence sees, and (query, key) pairs."""
    keys = pairs = 0
    w, s = case["window"], case["sinks"]
    for n, c in zip(*_prompt_lengths(case)):
        first = c - n
        lo = max(0, first - w + 1) if w else 0
        keys += c - lo + min(lo, s)
        if w:
            for p in range(first, c):
                lo = max(0, p - w + 1)
                pairs += p + 1 - lo + min(lo, s)
        else:
            pairs += n * first + n * (n + 1) // 2
    return keys, pairs


def work(case):
    op = case["op"]
    if op == "draft":
        _, new = _draft_lengths(case)
        T, B = sum(new) + case["slack"], case["batch"]
        return dict(bytes=24 * T + 16 * B + 8 * (sum(new) // PAGE) + 16 * B, flops=8 * T)
    if op == "turnover":
        held, kept, new = _turnover_lengths(case)
        T, B = sum(new) + case["slack"], case["batch"]
        pages = sum((n + PAGE - 1) // PAGE for n, k in zip(held, kept) if k == 0)
        return dict(bytes=24 * T + 32 * B + 16 * pages, flops=8 * T)
    if op == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return dict(bytes=4 * n + 8 * case["tokens"] * case["axes"], flops=3 * n)
    keys, pairs = _visible(case)
    q = sum(_prompt_lengths(case)[0]) * case["heads"] * case["dim"]
    return dict(bytes=4 * keys * case["kv_heads"] * case["dim"] + 4 * q,
                flops=4 * pairs * case["heads"] * case["dim"])


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prefix(x):
    got = [0]
    for n in x:
        got.append(got[-1] + n)
    return got


def _pool(g, lens, width, spare):
    """A block table for sequences that hold `lens` tokens, -1 elsewhere, and
    the stack of the other pages, all in random order."""
    pages = torch.tensor([(n + PAGE - 1) // PAGE for n in lens], device="cuda")
    held = int(pages.sum())
    order = torch.randperm(held + spare, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")[None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[col < pages[:, None]] = order[:held]
    free = torch.full((held + spare,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = order[held:]
    return dict(block_table=table, free_pages=free, free_count=_i32([spare]))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "draft":
        cached, new = _draft_lengths(case)
        width = (max(c + n for c, n in zip(cached, new)) + PAGE - 1) // PAGE + 1
        spare = sum((c + n + PAGE - 1) // PAGE - (c + PAGE - 1) // PAGE
                    for c, n in zip(cached, new)) + 5
        return dict(op=op, cached=_i32(cached), new=_i32(new),
                    num_tokens=max(1, sum(new) + case["slack"]), **_pool(g, cached, width, spare))
    if op == "turnover":
        held, kept, new = _turnover_lengths(case)
        width = (max(held) + PAGE - 1) // PAGE
        return dict(op=op, held=_i32(held), kept=_i32(kept), new=_i32(new),
                    num_tokens=sum(new) + case["slack"], **_pool(g, held, width, 5))
    if op == "rope":
        return dict(op=op, **_prepare_rope(case, g))
    return dict(op=op, **_prepare_prompt(case, g))


def _sections(case):
    """Pairs of each axis: unequal ones, their sum half the rotated width."""
    half, n = case["rotary"] // 2, case["axes"]
    part = half // n
    if n == 1:
        return [half]
    if n == 2:
        return [part, half - part]
    return [half - 2 * part + 2, part - 1, part - 1]


def _prepare_rope(case, g):
    T, Hq, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dt, half = DTYPES[case["dtype"]], case["rotary"] // 2
    # positions: text, then frames of 18 x 31 patches, then text again
    t = torch.arange(T, device="cuda")
    offset = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
    rows, cols = 18, 31
    grid = [t // (rows * cols), t // cols % rows, t % cols][3 - case["axes"]:]
    image = (t >= T // 8) & (t < T - T // 8)
    base = T // 8
    pos = [torch.where(image, base + x, t) + offset if case["axes"] > 1 else t + offset
           for x in grid]
    positions = torch.stack(pos).to(torch.int64)
    if case["axes"] == 1:
        positions = positions[0]
    max_pos = T + 1100
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    if case["fused"]:
        x = _randn(g, T, Hq + 2 * Hk, D).to(dt)
        q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    else:
        q, k = _randn(g, T, Hq, D).to(dt), _randn(g, T, Hk, D).to(dt)
    return dict(q=q, k=k, positions=positions.contiguous(), cos=angle.cos().float(),
                sin=angle.sin().float(), style=case["style"], sections=_sections(case),
                interleaved=case["order"] == "interleaved")


def _prepare_prompt(case, g):
    qs, ks = _prompt_lengths(case)
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    dt = DTYPES[case["dtype"]]
    slack = case["slack"]
    Tq, Tk = sum(qs) + slack, sum(ks) + slack
    lean = _randn(g, Hk, D)
    k = _randn(g, Tk, Hk, D)
    starts = _prefix(ks)
    k[torch.tensor(starts[:-1], device="cuda")] = lean * 1.5  # first tokens draw attention
    v = _randn(g, Tk, Hk, D) * torch.exp2(_randn(g, Tk, 1, 1) * 0.5)
    q = _randn(g, Tq, Hk, Hq // Hk, D) + 0.5 * lean[None, :, None]
    whole = case["context"] == 0
    return dict(q=q.reshape(Tq, Hq, D).to(dt), k=k.to(dt), v=v.to(dt), q_starts=_i32(_prefix(qs)),
                max_q=max(qs), k_starts=None if whole else _i32(starts), max_k=max(ks),
                window=case["window"], sinks=case["sinks"],
                out=torch.zeros(Tq, Hq, D, dtype=dt, device="cuda"),
                lse=torch.zeros(Tq, Hq, device="cuda"))


# --------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    return {"draft": _plain_draft, "turnover": _plain_turnover, "rope": _plain_rope,
            "prompt": _plain_prompt}[s["op"]](s)


def _run_own(s):
    from fp4_sparse_attention_fp4idx_gb300 import fp4idx as F
    op = s["op"]
    if op == "rope":
        q, k = F.rope_qk(s["q"], s["k"], s["positions"], s["cos"], s["sin"],
                         rope_style=s["style"], sections=s["sections"],
                         interleaved_axes=s["interleaved"])
        return dict(q=q, k=k)
    if op == "prompt":
        out, lse = F.prompt_attention(s["q"], s["k"], s["v"], s["q_starts"], s["max_q"],
                                      k_starts=s["k_starts"], max_k=s["max_k"],
                                      window=s["window"], sinks=s["sinks"], out=s["out"],
                                      lse=s["lse"])
        return dict(out=out, lse=lse)
    pool = (s["block_table"], s["free_pages"], s["free_count"])
    if op == "draft":
        maps = F.batch_extend(s["cached"], s["new"], *pool, s["num_tokens"])
        F.pages_release(maps.context_lens, s["cached"], *pool)
    else:
        F.pages_release(s["held"], s["kept"], *pool)
        maps = F.batch_extend(s["kept"], s["new"], *pool, s["num_tokens"])
    return dict(maps._asdict(), block_table=s["block_table"], free_pages=s["free_pages"],
                free_count=s["free_count"])


# -------- pages and maps
def _plain_extend(cached, new, table, free, count, num_tokens):
    """Takes pages for `new` tokens behind `cached` ones and maps the tokens.
    A sequence is served if its pages (and those of the sequences before it)
    are there, fit its row, and its tokens fit the step."""
    old, add = cached.long().clamp(min=0), new.long().clamp(min=0)
    has, want = (old + PAGE - 1) // PAGE, (old + add + PAGE - 1) // PAGE
    ends = add.cumsum(0)
    fits = (want <= table.shape[1]) & (ends <= num_tokens)
    need = torch.where(fits, want - has, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= count))
    starts = torch.cat([torch.zeros_like(ends[:1]), ends.clamp(max=num_tokens)])
    # pages
    col = torch.arange(table.shape[1], device="cuda")[None]
    fresh = served[:, None] & (col >= has[:, None]) & (col < want[:, None])
    at = count.long() - 1 - (upto - need)[:, None] - (col - has[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, len(free) - 1)], table))
    count.sub_((torch.where(served, need, 0)).sum().to(torch.int32))
    # tokens
    t = torch.arange(num_tokens, device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    seq = b.clamp(max=len(ends) - 1)
    real = (b < len(ends)) & served[seq]
    pos = torch.where(real, old[seq] + t - starts[seq], 0)
    page = table[seq, (pos // PAGE).clamp(max=table.shape[1] - 1)].long()
    return dict(q_starts=starts.to(torch.int32),
                context_lens=torch.where(served, old + add, old).to(torch.int32),
                slot_mapping=torch.where(real, page * PAGE + pos % PAGE, -1), positions=pos,
                seq_ids=torch.where(b < len(ends), b, 0).to(torch.int32),
                row_lens=torch.where(real, pos + 1, 0).to(torch.int32))


def _plain_release(held, kept, table, free, count):
    """Gives back the pages behind `kept` tokens, the last one first."""
    held = held.long().clamp(min=0)
    has = ((held + PAGE - 1) // PAGE).clamp(max=table.shape[1])
    keep = (torch.minimum(kept.long().clamp(min=0), held) + PAGE - 1) // PAGE
    col = torch.arange(table.shape[1], device="cuda")[None]
    gone = (col >= keep[:, None]) & (col < has[:, None])
    n = gone.sum()
    rank = gone.flatten().cumsum(0).view(gone.shape) - 1
    at = torch.where(gone, count.long() + n - 1 - rank, len(free))
    longer = torch.cat([free, free[:1]])
    longer[at.flatten()] = table.flatten()
    free.copy_(longer[:-1])
    count.add_(n.to(torch.int32))
    table.masked_fill_(gone, -1)


def _plain_draft(s):
    pool = (s["block_table"], s["free_pages"], s["free_count"])
    maps = _plain_extend(s["cached"], s["new"], *pool, s["num_tokens"])
    _plain_release(maps["context_lens"], s["cached"], *pool)
    return dict(maps, block_table=pool[0], free_pages=pool[1], free_count=pool[2])


def _plain_turnover(s):
    pool = (s["block_table"], s["free_pages"], s["free_count"])
    _plain_release(s["held"], s["kept"], *pool)
    maps = _plain_extend(s["kept"], s["new"], *pool, s["num_tokens"])
    return dict(maps, block_table=pool[0], free_pages=pool[1], free_count=pool[2])


# -------- rotary positions
def _axis_of_pair(sections, interleaved):
    """The axis whose position turns each pair: ranges of pairs, or pair i by
    axis i % n while that axis has pairs left, else by axis 0."""
    n, half = len(sections), sum(sections)
    if not interleaved:
        return [a for a, m in enumerate(sections) for _ in range(m)]
    return [i % n if i // n < sections[i % n] else 0 for i in range(half)]


def _plain_rope(s):
    half = s["cos"].shape[1]
    pos = s["positions"].view(-1, s["q"].shape[0])
    axis = torch.tensor(_axis_of_pair(s["sections"], s["interleaved"])).cuda()
    col = torch.arange(half, device="cuda")
    at = pos[axis].t()  # [T, half]
    c, d = s["cos"][at, col][:, None], s["sin"][at, col][:, None]

    def turn(x):
        y = x.float()
        r = y[..., :2 * half]
        if s["style"] == "neox":
            a, b = r[..., :half], r[..., half:]
            got = torch.cat([a * c - b * d, b * c + a * d], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            got = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
        return torch.cat([got, y[..., 2 * half:]], -1).to(x.dtype)

    return dict(q=turn(s["q"]), k=turn(s["k"]))


# -------- attention of packed prompts
def _plain_prompt(s):
    """Padded to the longest sequence where the batch's scores fit a few GB at
    a time: blocks of query rows, one key head after another."""
    q, k, v = s["q"], s["k"], s["v"]
    (Tq, Hq, D), (Tk, Hk, _) = q.shape, k.shape
    G, M, N = Hq // Hk, s["max_q"], s["max_k"]
    qst = s["q_starts"].long()
    kst = s["k_starts"].long() if s["k_starts"] is not None else qst
    B = len(qst) - 1
    n, c = qst[1:] - qst[:-1], kst[1:] - kst[:-1]
    key = torch.arange(N, device="cuda")
    kat = (kst[:-1, None] + key).clamp(max=Tk - 1)
    held = key[None] < c[:, None]
    rows = max(1, min(M, (1 << 29) // (B * G * N)))
    for h in range(Hk):
        kp = k[:, h][kat].float().transpose(1, 2)  # B, D, N
        vp = v[:, h][kat].float().masked_fill_(~held[..., None], 0.0)
        for a in range(0, M, rows):
            i = torch.arange(a, min(M, a + rows), device="cuda")
            m = len(i)
            real = i[None] < n[:, None]
            at = (qst[:-1, None] + i).clamp(max=Tq - 1)
            x = q[at, h * G:(h + 1) * G].float().transpose(1, 2).reshape(B, G * m, D)
            x = torch.matmul(x, kp).view(B, G, m, N)
            x *= 1.0 / math.sqrt(D)
            pos = ((c - n)[:, None] + i)[..., None]  # B, m, 1
            seen = (key <= pos) & held[:, None]
            if s["window"]:
                seen = seen & ((key > pos - s["window"]) | (key < s["sinks"]))
            x.masked_fill_(~seen[:, None], NEG)
            top = x.amax(-1, keepdim=True)
            top = torch.where(top == NEG, 0.0, top)
            p = x.sub_(top).exp_()
            den = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(B, G * m, N), vp).view(B, G, m, D)
            o = o / torch.where(den == 0, 1.0, den)
            e = torch.where(den == 0, NEG, den.log() + top).squeeze(-1)
            # rows that are not there go to a row behind the output
            to = torch.where(real, at, Tq)
            for dst, src in ((s["out"], o.permute(0, 2, 1, 3)), (s["lse"], e.permute(0, 2, 1))):
                part = torch.cat([dst[:, h * G:(h + 1) * G], dst[:1, :G]])
                part[to.flatten()] = src.reshape(B * m, *part.shape[1:]).to(dst.dtype)
                dst[:, h * G:(h + 1) * G] = part[:-1]
    return dict(out=s["out"], lse=s["lse"])


# ------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] in ("draft", "turnover"):
        return None  # whole numbers: compared for equality
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_prompt(case, s)


def _exact_rope(s):
    """Each pair as a complex number, multiplied by its axis's turn."""
    half = s["cos"].shape[1]
    pos = s["positions"].view(-1, s["q"].shape[0])
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    n, left = len(s["sections"]), list(s["sections"])
    cols, a = [], 0
    for i in range(half):
        if s["interleaved"]:
            axis = i % n if left[i % n] > i // n else 0
        else:
            while left[a] == 0:
                a += 1
            left[a] -= 1
            axis = a
        cols.append(turn[pos[axis], i])
    z = torch.stack(cols, -1)[:, None]
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        if s["style"] == "neox":
            first, second = slice(0, half), slice(half, 2 * half)
        else:
            first, second = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
        w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
        x[..., first], x[..., second] = w.real, w.imag
        got[name] = x
    return got


def _exact_prompt(case, s):
    qs, ks = _prompt_lengths(case)
    G, D = case["heads"] // case["kv_heads"], case["dim"]
    out, lse = s["out"].double(), s["lse"].double()
    w, sinks = case["window"], case["sinks"]
    qa = ka = 0
    for n, c in zip(qs, ks):
        first = c - n
        for h in range(case["kv_heads"]):
            k, v = s["k"][ka:ka + c, h].double(), s["v"][ka:ka + c, h].double()
            step = max(1, (1 << 27) // (G * c))
            for a in range(0, n, step):
                b = min(n, a + step)
                end = first + b  # keys behind the block's last query are not seen
                p = torch.arange(first + a, end, device="cuda").repeat_interleave(G)[:, None]
                key = torch.arange(end, device="cuda")[None]
                x = s["q"][qa + a:qa + b, h * G:(h + 1) * G].double().reshape(-1, D) @ k[:end].T
                x /= math.sqrt(D)
                hidden = key > p
                if w:
                    hidden |= (p - key >= w) & (key >= sinks)
                x.masked_fill_(hidden, NEG)
                e = torch.logsumexp(x, -1)
                x = x.sub_(e[:, None]).exp_()
                out[qa + a:qa + b, h * G:(h + 1) * G] = (x @ v[:end]).view(b - a, G, D)
                lse[qa + a:qa + b, h * G:(h + 1) * G] = e.view(b - a, G)
        qa, ka = qa + n, ka + c
    return dict(out=out, lse=lse)
