"""Plain definitions of the step operators (include/fp4idx_step.h) and the error
bounds that their tests hold the kernels to.  Loops over sequences and heads, in
whole numbers or 64 bits; shares no code with the library."""
from __future__ import annotations

import math

import torch

PAGE = 64


def pages(n):
    return (n + PAGE - 1) // PAGE


def extend(cached, new, table, free, count, T):
    """(maps dict of lists, table, free count, whether a sequence was not served)
    by a loop; the arguments are lists and stay as they are."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    count0 = count = min(max(count, 0), len(free))
    asked, at, full = 0, 0, False
    m = dict(q_starts=[], context_lens=[], slot_mapping=[-1] * T, positions=[0] * T,
             seq_ids=[0] * T, row_lens=[0] * T)
    for b, (old, add) in enumerate(zip(cached, new)):
        old, add = max(old, 0), max(add, 0)
        has, want = pages(old), pages(old + add)
        fits = want <= width and at + add <= T
        need = want - has if fits else 0
        served = fits and (need == 0 or asked + need <= count0)
        m["q_starts"].append(min(at, T))
        m["context_lens"].append(old + add if served else old)
        if served:
            for j in range(need):
                table[b][has + j] = free[count0 - 1 - asked - j]
            if need:
                count = count0 - asked - need
        full = full or not served
        asked += need
        for i in range(add):
            t = at + i
            if t >= T:
                break
            m["seq_ids"][t] = b
            if served:
                p = old + i
                m["slot_mapping"][t] = table[b][p // PAGE] * PAGE + p % PAGE
                m["positions"][t] = p
                m["row_lens"][t] = p + 1
        at += add
    m["q_starts"].append(min(at, T))
    return m, table, count, full


def release(held, kept, table, free, count):
    """(table, free list, count, whether a page found no place)."""
    table, free = [list(r) for r in table], list(free)
    width = len(table[0]) if table else 0
    count = min(max(count, 0), len(free))
    gone = []
    for b, (h, k) in enumerate(zip(held, kept)):
        h = max(h, 0)
        k = min(max(k, 0), h)
        for p in range(pages(k), min(pages(h), width)):
            gone.append(table[b][p])
            table[b][p] = -1
    for i, page in enumerate(reversed(gone)):
        if count + i < len(free):
            free[count + i] = page
    full = count + len(gone) > len(free)
    return table, free, min(count + len(gone), len(free)), full


def axis_of_pair(sections, interleaved):
    n, half = len(sections), sum(sections)
    if interleaved:
        return [i % n if i // n < sections[i % n] else 0 for i in range(half)]
    return [a for a, m in enumerate(sections) for _ in range(m)]


def rope(x, positions, cos, sin, sections, interleaved, neox, dtype):
    """The rows of x [T, H, D] turned, in `dtype`, and the sum of the magnitudes that
    each element is made of.  positions [axes, T]."""
    half = cos.shape[1]
    axis = torch.tensor(axis_of_pair(sections, interleaved), device=x.device)
    at = positions[axis].t()  # [T, half]
    col = torch.arange(half, device=x.device)
    c, s = cos[at, col].to(dtype)[:, None], sin[at, col].to(dtype)[:, None]
    y, mag = x.to(dtype).clone(), x.to(dtype).abs()
    first, second = (slice(0, half), slice(half, 2 * half)) if neox else \
        (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = (a * c).abs() + (b * s).abs()
    mag[..., second] = (b * c).abs() + (a * s).abs()
    return y, mag


def attend(q, k, v, qs, ks, window, sinks, scale, max_k=None):
    """out, lse (doubles, zero and -inf for rows in no sequence) and, per row, what
    the bounds are made of: sum p|v|, sum |v|, the largest sum |q k| * scale, keys."""
    T, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    dev = q.device
    z = torch.zeros(T, H, D, dtype=torch.float64, device=dev)
    out, pv, sv = z, z.clone(), z.clone()
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    top = torch.zeros(T, H, dtype=torch.float64, device=dev)
    keys = torch.zeros(T, H, dtype=torch.float64, device=dev)
    for b in range(len(qs) - 1):
        a, n, ka, c = qs[b], qs[b + 1] - qs[b], ks[b], ks[b + 1] - ks[b]
        if n <= 0 or c <= 0:
            continue
        first, held = c - n, c if max_k is None else min(c, max_k)
        if held <= 0:
            continue
        at = torch.arange(held, device=dev)[None]
        pos = (first + torch.arange(n, device=dev)).repeat_interleave(G)[:, None]
        seen = at <= pos
        if window:
            seen = seen & ((at > pos - window) | (at < sinks))
        for h in range(Hk):
            sl = slice(h * G, (h + 1) * G)
            qq = q[a:a + n, sl].double().reshape(n * G, D)
            kk, vv = k[ka:ka + held, h].double(), v[ka:ka + held, h].double()
            x = torch.where(seen, (qq @ kk.T) * scale, -math.inf)
            e = torch.logsumexp(x, -1)
            p = torch.where(seen, torch.exp(x - torch.where(e == -math.inf, 0.0, e)[:, None]), 0.0)
            mag = torch.where(seen, (qq.abs() @ kk.abs().T) * abs(scale), 0.0).amax(-1)
            for dst, got in ((out, p @ vv), (lse, e), (pv, p @ vv.abs()),
                             (sv, seen.double() @ vv.abs()), (top, mag),
                             (keys, seen.sum(-1).double())):
                dst[a:a + n, sl] = got.reshape(n, G, *got.shape[1:])
    return out, lse, pv, sv, top, keys


def check(out, lse, ref):
    """Holds out / lse to attend()'s.

    A score is a sum of <= 128 exact products in fp32 (each partial sum within
    2^-24 of sum|q k|, at most 2^-17 in all, doubled for the tensor core's
    truncating alignment) and is scaled once (2^-23 of itself, within that);
    ex2.approx, log2 and the references' differences add less than 2^-19.  A
    probability is rounded to the elements' type, by eps / 2 of itself, or, in
    fp16, by half the least subnormal, 2^-25, where the row's largest is at least
    2^10 (2^-35; in bf16 nothing above 2^-126 vanishes).  The sums: at most 40
    additions in a tile of 128 keys and one for each tile (probabilities), one for
    16 keys (outputs, 2^-23 each with the truncation).  The output is rounded once."""
    o, e, pv, sv, top, keys = ref
    u = torch.finfo(out.dtype).eps / 2
    d_score = 2.0 ** -16 * top + 2.0 ** -19
    sums = (40 + keys / 128) * 2.0 ** -24
    products = (8 + keys / 16) * 2.0 ** -23
    least = 2.0 ** -34 if out.dtype == torch.float16 else 2.0 ** -120
    rel = (u + 2 * d_score + sums + products)[..., None]
    tol = u * o.abs() + (1 + u) * (pv * rel + least * sv) + torch.finfo(out.dtype).tiny * u
    err = (out.double() - o).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err - tol).max()), float(err.max()))
    empty = e == -math.inf
    assert torch.equal(torch.isneginf(lse), empty)
    lerr = (lse.double() - e).abs()[~empty]
    ltol = (d_score + sums + 2.0 ** -19 * (1 + e.abs()))[~empty]
    assert bool((lerr <= ltol).all()), float((lerr - ltol).max())
    assert bool((out[empty] == 0).all())
