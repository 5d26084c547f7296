"""The operators of hybrid stacks in 64 bits, a request after the other, with the sums of the terms' absolute values
that the tests' error bounds are made of."""
import math

import torch


def f64(t):
    return None if t is None else t.detach().double()


def conv(x, weight, bias, cache, slots, positions, spans, silu, kept):
    """x [rows, channels] of the spans [(begin, end)], slots a list (None: no cache; negative: no slot), positions a
    list; kept: inputs stored at most.  Returns (y, error sums, cache): y of rows in no span is 0."""
    W = weight.shape[1]
    x, weight, bias = f64(x), f64(weight), f64(bias)
    y, m = torch.zeros_like(x), torch.zeros_like(x)
    cache = None if cache is None else cache.clone()
    for i, (a, b) in enumerate(spans):
        if a == b:
            continue
        slot = -1 if cache is None else slots[i]
        p = 0 if slot < 0 else positions[i]
        past = torch.zeros(W - 1, x.shape[1], dtype=torch.float64, device=x.device)
        if slot >= 0:
            R = cache.shape[1]
            for j in range(1, W):
                if p >= j:
                    past[W - 1 - j] = cache[slot, (p - j) % R].double()
        line = torch.cat([past, x[a:b]])
        v = torch.zeros(b - a, x.shape[1], dtype=torch.float64, device=x.device)
        if bias is not None:
            v += bias
        mm = v.abs()
        for j in range(W):
            v = v + line[j:j + b - a] * weight[:, j]
            mm = mm + (line[j:j + b - a] * weight[:, j]).abs()
        y[a:b], m[a:b] = (v * torch.sigmoid(v) if silu else v), mm
        if slot >= 0:
            for t in range(max(a, b - kept), b):
                cache[slot, (p + t - a) % R] = x[t].to(cache.dtype)
    return y, m, cache


def rotate(v, positions, freq, interleaved, amplitude):
    """(turned, sums) of v [tokens, heads, dim] at positions [tokens]."""
    v, n = f64(v), freq.numel()
    angle = positions.double()[:, None] * f64(freq)
    c, s = (amplitude * angle.cos())[:, None], (amplitude * angle.sin())[:, None]
    out, m = v.clone(), v.abs()
    ia = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    ib = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    a, b = v[..., ia], v[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    m[..., ia] = m[..., ib] = abs(amplitude) * (a.abs() + b.abs())
    return out, m


def attention(q, k_cache, v_cache, page_table, lengths, scale):
    """(y, sums of |weight v|, relative error of a weight from a unit of the scores' rounding: see the caller) of
    q [batch, window, H, dim]; requests of length 0 and bad lengths are the caller's business (given as 0)."""
    b, T, H, dim = q.shape
    pages, page, G = k_cache.shape[:3]
    y = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    m, top = torch.zeros_like(y), torch.zeros(b, T, H, 1, dtype=torch.float64, device=q.device)
    for r, n in enumerate(lengths):
        if n == 0:
            continue
        at = torch.arange(n, device=q.device)
        where = page_table[r, at // page].long()
        good = (where >= 0) & (where < pages)
        where = where.clamp(0, pages - 1)
        k = f64(k_cache[where, at % page]).repeat_interleave(H // G, 1)  # [n, H, dim]
        v = f64(v_cache[where, at % page]).repeat_interleave(H // G, 1)
        for t in range(T):
            see = good & (at <= n - T + t)
            if not bool(see.any()):
                continue
            qq, kk, vv = f64(q[r, t]), k[see], v[see]
            s = (kk * qq).sum(-1) * scale                 # [n, H]
            w = torch.softmax(s, 0)[..., None]
            y[r, t], m[r, t] = (w * vv).sum(0), (w * vv.abs()).sum(0)
            top[r, t, :, 0] = (kk.abs() * qq.abs()).sum(-1).amax(0) * abs(scale)
    return y, m, top


def table(lengths, page, width, gen):
    """(page table, pages) for the lengths: pages in random order, -1 where none is needed, two pages nobody's."""
    need = [-(-n // page) for n in lengths]
    free = (2 + torch.randperm(sum(need), generator=gen)).tolist()
    t = torch.full((len(lengths), max(width, max(need, default=0), 1)), -1, dtype=torch.int32)
    for r, n in enumerate(need):
        for i in range(n):
            t[r, i] = free.pop()
    return t.cuda(), sum(need) + 2


def ceil_log2(n):
    return math.ceil(math.log2(max(n, 1)))
