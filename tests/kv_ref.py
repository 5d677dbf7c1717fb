"""64-bit definitions of the 8-bit cache operators (include/fp4idx_attention.h)
and of the error bounds that their tests hold the kernels to.  Plain loops over
sequences and heads; shares no code with the library."""
from __future__ import annotations

import math

import torch

PAGE = 64
NAN_CODE = 0x7F


def pow2(e):
    """2^e as a double, e an integer tensor."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def e4m3_round(x):
    """The nearest E4M3 value of each double, ties to even, saturating."""
    _, e = torch.frexp(x)
    step = pow2((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def block_scale(amax):
    """ceil_pow2(max(amax / 448, 2^-126)) of a double tensor."""
    m, e = torch.frexp((amax / 448).clamp(min=2.0 ** -126))
    return pow2(torch.where(m == 0.5, e - 1, e))


def codes_value(codes):
    return codes.view(torch.uint8).view(torch.float8_e4m3fn).double()


def store(x, slots, codes, scale):
    """The expected code values (double) and scales after a store of x
    [T, H, D]; codes uint8 [B, H, 64, D] and scale [B, H] before it."""
    val, sc = codes_value(codes), scale.double()
    slots = slots.tolist()
    t = 0
    while t < len(slots):
        s = slots[t]
        if s < 0 or s >= codes.shape[0] * PAGE:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % PAGE:
            n += 1
        page, off = s // PAGE, s % PAGE
        rows = x[t:t + n].double().transpose(0, 1)  # [H, n, D]
        now = block_scale(rows.abs().amax((1, 2)))
        if off > 0:
            old = sc[page]
            now = torch.maximum(now, old)
            grown = now > old
            kept = e4m3_round(val[page, :, :off] * (old / now)[:, None, None])
            val[page, :, :off] = torch.where(grown[:, None, None], kept, val[page, :, :off])
        val[page, :, off:off + n] = e4m3_round(rows / now[:, None, None])
        sc[page] = now
        t += n
    return val, sc


def rows_of(codes, scale, table_row, positions):
    """Values (double) [n, H, D] at the positions of one sequence."""
    page, off = table_row[positions // PAGE].long(), positions % PAGE
    return codes_value(codes[page, :, off]) * scale[page].double()[..., None]


def attend(q, k, v, seen, scale):
    """One kv head: q [m, D], k, v [n, D] doubles, seen [m, n].  Returns out,
    lse, sum p|v| and the largest sum |q k| * scale of each row."""
    x = torch.where(seen, (q @ k.T) * scale, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.where(seen, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    mag = torch.where(seen, (q.abs() @ k.abs().T) * abs(scale), 0.0)
    top = mag.amax(-1) if k.shape[0] else torch.zeros(q.shape[0], dtype=q.dtype, device=q.device)
    return p @ v, lse, p @ v.abs(), top


def check(out, lse, ref, n):
    """Holds out / lse to the bounds (ref = attend's four, rows flattened).

    A score is a sum of <= 128 exact products in fp32 (each partial sum within
    2^-24 of sum|q k|, at most 2^-17 in all, doubled for the tensor core's
    truncating alignment), a probability is rounded to fp16 (2^-11 of itself;
    or half the least subnormal, 2^-25, of a scale where the row's largest
    contribution is at least 2^10, times a code of at most 448: taken here as
    2^-34 * 448 of max sum p|v| over d),
    ex2.approx and the fp32 sums add less than 2^-19, and the output is rounded
    once to its type."""
    o, e, pv, top = ref
    u = torch.finfo(out.dtype).eps / 2
    d_score = 2.0 ** -16 * top + 2.0 ** -19
    tiny = 2.0 ** -34 * 448 * n * pv.amax(-1, keepdim=True) + torch.finfo(out.dtype).tiny * u
    tol = u * o.abs() + (1 + u) * (pv * (2.0 ** -11 + 2 * d_score[:, None]) + tiny)
    err = (out.double() - o).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err - tol).max()), float(err.max()))
    empty = e == -math.inf
    assert torch.equal(torch.isneginf(lse), empty)
    ok = ~empty
    lerr = (lse.double() - e).abs()[ok]
    ltol = (d_score + 2.0 ** -19 * (1 + e.abs()))[ok]
    assert bool((lerr <= ltol).all()), float((lerr - ltol).max())
    assert bool((out[empty] == 0).all())


def dense(q, cache, table, ctx, starts, window, sinks, scale):
    """attend()'s four for every (token, head) of a ragged batch."""
    kc, vc, ks, vs = cache
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    z = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    o, pv = z, z.clone()
    e = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    top = torch.zeros(T, Hq, dtype=torch.float64, device=q.device)
    for b, c in enumerate(ctx):
        a, n = starts[b], starts[b + 1] - starts[b]
        if n == 0 or c == 0:
            continue
        at = torch.arange(c, device=q.device)
        k, v = rows_of(kc, ks, table[b], at), rows_of(vc, vs, table[b], at)
        pos = torch.arange(c - n, c, device=q.device).repeat_interleave(G)[:, None]
        seen = at[None] <= pos
        if window:
            seen = seen & ((at[None] > pos - window) | (at[None] < sinks))
        for h in range(Hkv):
            sl = slice(h * G, (h + 1) * G)
            got = attend(q[a:a + n, sl].double().reshape(n * G, D), k[:, h], v[:, h], seen, scale)
            for dst, x in zip((o, e, pv, top), got):
                dst[a:a + n, sl] = x.reshape(n, G, *x.shape[1:])
    return o.view(-1, D), e.view(-1), pv.view(-1, D), top.view(-1)


def sparse(q, cache, table, indices, seq_ids, scale):
    kc, vc, ks, vs = cache
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    got = []
    for t in range(T):
        at = indices[t].long()
        at = at[at >= 0]
        k = rows_of(kc, ks, table[seq_ids[t]], at)
        v = rows_of(vc, vs, table[seq_ids[t]], at)
        for h in range(Hkv):
            seen = torch.ones(G, len(at), dtype=torch.bool, device=q.device)
            got.append(attend(q[t, h * G:(h + 1) * G].double(), k[:, h], v[:, h], seen, scale))
    return tuple(torch.cat([g[i] for g in got]) for i in range(4))


def topk(logits, k, lens):
    """Indices [R, k] and counts by sorting (value descending, index
    ascending) in Python."""
    R, N = logits.shape
    ind = torch.full((R, k), -1, dtype=torch.int32)
    cnt = torch.zeros(R, dtype=torch.int32)
    rows = logits.double().cpu().tolist()
    for r in range(R):
        n = min(max(int(lens[r]), 0), N)
        cand = [(-rows[r][i] + 0.0, i) for i in range(n)
                if rows[r][i] > -math.inf and rows[r][i] == rows[r][i]]
        cand.sort()
        sel = sorted(i for _, i in cand[:k])
        ind[r, :len(sel)] = torch.tensor(sel, dtype=torch.int32)
        cnt[r] = len(sel)
    return ind, cnt


def make_cache(g, blocks, heads, dim, spread=0.5, device="cuda"):
    """Random codes and scales of two filled caches (keys, values)."""
    out = []
    for _ in range(2):
        x = torch.randn(blocks, heads, PAGE, dim, generator=g, device=device, dtype=torch.float64)
        x = x * torch.exp2(torch.randn(blocks, heads, 1, 1, generator=g, device=device,
                                       dtype=torch.float64) * spread)
        s = block_scale(x.abs().amax((2, 3)))
        c = (x / s[..., None, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        out += [c, s.float()]
    kc, ks, vc, vs = out
    return kc, vc, ks, vs


def make_table(g, ctx, blocks, device="cuda"):
    width = max(1, max((c + PAGE - 1) // PAGE for c in ctx) if ctx else 1)
    order = torch.randperm(blocks, generator=g, device=device).to(torch.int32)
    table = torch.full((len(ctx), width), -7, dtype=torch.int32, device=device)
    at = 0
    for b, c in enumerate(ctx):
        n = (c + PAGE - 1) // PAGE
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= blocks
    return table
