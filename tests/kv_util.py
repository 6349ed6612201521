"""Plain implementations in 64 bits of the key-value cache's operators and of the
rotary positions, for the tests (numpy / torch, nothing of the library)."""

import math

import numpy as np
import torch

import mx4_util

HALF_BF16 = 2.0 ** -8   # half a step of BF16, relative


def pages_of(tokens, page):
    return -(-tokens // page)


def extend(table, lengths, counts, free, free_count, tokens, page):
    """offsets, lengths, slots, positions, free_count and the table afterwards (numpy)."""
    table = np.array(table)
    width, taken, spent, row = table.shape[1], 0, 0, 0
    pages = len(free)
    free_count = min(max(int(free_count), 0), pages)
    offsets, out = [], []
    slots, positions = np.full(tokens, -1, np.int32), np.zeros(tokens, np.int32)
    for b, (past, new) in enumerate(zip(lengths.tolist(), counts.tolist())):
        past, new = max(past, 0), max(new, 0)
        offsets.append(min(row, tokens))
        fits = row + new <= tokens and past + new < 2 ** 31 - 1 and pages_of(past + new, page) <= width
        held = pages_of(past, page)
        need = pages_of(past + new, page) - held if fits else 0
        granted = fits and (need == 0 or taken + need <= free_count)
        if granted:
            for j in range(need):
                table[b, held + j] = free[free_count - 1 - (taken + j)]
            if need:
                spent = taken + need
        taken += need
        for i in range(new):
            if row + i < tokens:
                positions[row + i] = min(past + i, 2 ** 31 - 1)
                if granted:
                    p = table[b, (past + i) // page]
                    slots[row + i] = p * page + (past + i) % page if 0 <= p < pages else -1
        out.append(past + new if granted else past)
        row += new
    offsets.append(min(row, tokens))
    return (np.array(offsets, np.int32), np.array(out, np.int32), slots, positions,
            np.array([free_count - spent], np.int32), table)


def release(table, lengths, finished, free, free_count, page):
    table, free, n = np.array(table), np.array(free), int(free_count)
    lengths = np.maximum(lengths, 0)
    for b in np.flatnonzero(finished):
        for j in range(min(pages_of(int(lengths[b]), page), table.shape[1])):
            if 0 <= table[b, j] < len(free) and n < len(free):
                free[n] = table[b, j]
                n += 1
            table[b, j] = -1
    return np.where(finished, 0, lengths).astype(np.int32), np.array([n], np.int32), table, free


def cache_bytes(k, v):
    """The cache's records of BF16 bit patterns k, v [pages, heads, page, D] (numpy)."""
    n, h, p, d = k.shape

    def quantize(x):
        codes, scales = mx4_util.quantize(x.reshape(-1, d))
        return codes.reshape(n, h, p, d // 2), scales.reshape(n, h, p, d // 32)
    (kc, ks), (vc, vs) = quantize(k), quantize(v)
    vc = vc.reshape(n, h, p // 4, 4, d // 8, 4).transpose(0, 1, 2, 4, 3, 5)
    return np.concatenate([np.ascontiguousarray(x).reshape(n, h, -1) for x in (kc, vc, ks, vs.transpose(0, 1, 3, 2))], 2)


def cache_values(cache, page, d):
    """k and v in 64 bits [pages, heads, page, D] of a cache (torch, on its device)."""
    n, h = cache.shape[:2]
    half, few = page * d // 2, page * d // 32
    kc, vc, ks, vs = cache.split((half, half, few, few), 2)
    vc = vc.reshape(n, h, page // 4, d // 8, 4, 4).transpose(3, 4).reshape(n, h, page, d // 2)
    vs = vs.reshape(n, h, d // 32, page).transpose(2, 3)
    table = torch.tensor(np.concatenate((mx4_util.E2M1, -mx4_util.E2M1)), device=cache.device)

    def values(codes, scales):
        c = torch.stack((codes & 15, codes >> 4), -1).reshape(n, h, page, d // 32, 32).long()
        return (table[c] * torch.exp2(scales.double() - 127)[..., None]).reshape(n, h, page, d)
    return values(kc.reshape(n, h, page, d // 2), ks.reshape(n, h, page, d // 32)), values(vc, vs)


def attention(q, k, v, page, table, lengths, offsets, scale, window):
    """(out, lse, bound of out, bound of lse) in 64 bits for values k, v [pages, heads,
    page, D]; rows of no sequence NaN.

    The bounds count roundings: the output's (half a step of BF16), each weight's
    (the same), and what a score may be off: the query's two parts hold it to 2^-21 of
    its row's largest value, and a sum of at most 512 products in fp32 is off by at most
    512 * 2^-24 of the sum of their magnitudes, as are the few operations behind it.  A
    weight p_j is then off by E of itself, and so is the sum that divides."""
    t, heads, d = q.shape
    hkv, pages = k.shape[1], k.shape[0]
    group = heads // hkv
    q = q.double()
    out, bound = torch.full((t, heads, d), math.nan, dtype=torch.float64, device=q.device), torch.zeros((t, heads, d), dtype=torch.float64, device=q.device)
    lse, lse_bound = torch.full((t, heads), math.nan, dtype=torch.float64, device=q.device), torch.zeros((t, heads), dtype=torch.float64, device=q.device)
    offsets = list(range(len(lengths) + 1)) if offsets is None else offsets
    for b, length in enumerate(lengths):
        i0, i1 = offsets[b], offsets[b + 1]
        n = i1 - i0
        if n <= 0:
            continue
        length = min(max(length, 0), table.shape[1] * page)
        ids = table[b, :pages_of(length, page)].long()
        there = ((ids >= 0) & (ids < pages)).repeat_interleave(page)[:length]
        ids = ids.clamp(0, pages - 1)
        key = torch.arange(length, device=q.device)
        at = torch.arange(length - n, length, device=q.device)[:, None]
        sees = (key <= at) & there
        if window:
            sees &= key > at - window
        for h in range(hkv):
            kk, vv = (x[ids, h].reshape(-1, d)[:length] for x in (k, v))
            vv = torch.where(sees.any(0)[:, None], vv, 0.0)
            kk = torch.where(sees.any(0)[:, None], kk, 0.0)
            for r in range(h * group, (h + 1) * group):
                x = q[i0:i1, r]
                s = (x @ kk.t()) * scale
                s = torch.where(sees, s, -math.inf)
                total = torch.logsumexp(s, 1, keepdim=True) if length else torch.full((n, 1), -math.inf, dtype=torch.float64, device=q.device)
                p = torch.where(sees, torch.exp(s - torch.where(torch.isinf(total), 0.0, total)), 0.0)
                o = p @ vv
                a = p @ vv.abs()
                off = scale * (x.abs().amax(1, keepdim=True) * 2.0 ** -21 * kk.abs().sum(1) + 2.0 ** -14 * (x.abs() @ kk.abs().t()))
                e = torch.where(sees, off, 0.0).amax(1, keepdim=True) + 2.0 ** -18 if length else torch.zeros((n, 1), dtype=torch.float64, device=q.device)
                out[i0:i1, r], lse[i0:i1, r] = o, total[:, 0]
                bound[i0:i1, r] = HALF_BF16 * o.abs() + (HALF_BF16 + 2 * e) * 1.01 * a + 1e-37
                lse_bound[i0:i1, r] = (e + 2.0 ** -20 * (1 + torch.where(torch.isinf(total), 0.0, total).abs()))[:, 0]
    return out, lse, bound, lse_bound


def rotate(x, positions, turns, magnitude, interleaved, inverse=False):
    """x [T, heads, D] turned, in 64 bits, and the sum of magnitudes of each result's terms."""
    n = turns.numel()
    t = torch.remainder(positions.double()[:, None, None] * turns.double(), 1.0)
    c, s = torch.cos(2 * math.pi * t) * magnitude, torch.sin(2 * math.pi * t) * magnitude
    if inverse:
        s = -s
    y, terms = x.double().clone(), x.double().abs()
    even, odd = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x.double()[..., even], x.double()[..., odd]
    y[..., even], y[..., odd] = a * c - b * s, a * s + b * c
    terms[..., even] = terms[..., odd] = (a.abs() + b.abs()) * abs(magnitude)
    return y, terms
