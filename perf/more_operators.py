"""Cases of the operators around a hybrid stack's caches: the short convolution
before the state space operator, and the attention layers between such blocks,
whose keys and values lie in pages.

  conv    causal_conv       packed prompts -> outputs, and the last inputs into the convolution's cache
  cstep   causal_conv_step  new tokens of running requests after their cached inputs, drafts among them
  rope    rotary_append     rotary positions on q and k of new tokens; k and v go to their pages
  attn    paged_attention   new tokens of running requests over the pages of their keys and values
  copy    copy_pages        pages of all layers' pools copied in one call: forks of shared prefixes, compaction

Channel counts are those of the package's own layers (80 heads of 64 with one
group of 128, 128 or 256 heads with eight: heads * 64 + 2 * groups * 128);
attention sizes are generic.
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one short prompt alone: a first token's latency
        dict(name="conv_1x37_c5376", op="conv", C=5376, width=4, R=4, seqs=1, tokens=37, longest=37, inputs="bf16",
             initial=False, bias=True, silu=True, sliced=True),
        # the next pieces of four long prompts: the first tokens look back into the cache
        dict(name="conv_4seq_8k_c18432", op="conv", C=18432, width=4, R=8, seqs=4, tokens=8192, longest=2560,
             inputs="bf16", initial=True, bias=True, silu=True, sliced=True),
        # a full batch decoding, one token each
        dict(name="cstep_256_c18432", op="cstep", C=18432, width=4, R=4, batch=256, T=1, inputs="bf16", pads=0,
             bias=True, silu=True, sliced=True),
        # drafts of four tokens, inputs in 32 bits, one request of the batch idle
        dict(name="cstep_16x4_c10240_f32", op="cstep", C=10240, width=4, R=11, batch=16, T=4, inputs="f32", pads=1,
             bias=True, silu=True, sliced=False),
        # one request's new token
        dict(name="rope_1_h32", op="rope", H=32, G=8, dim=128, rot=128, batch=1, T=1, page=16, far=3000, inputs="bf16",
             packed=0, longest=0, swap=False, amplitude=1.0, sliced=True, joined=False),
        # the next pieces of five long documents, half of each head rotated, neighbours paired, far positions
        dict(name="rope_5seq_8k_h32", op="rope", H=32, G=8, dim=128, rot=64, batch=5, T=0, page=64, far=500000,
             inputs="bf16", packed=8192, longest=3001, swap=True, amplitude=1.2, sliced=True, joined=True),
        # a few requests of a small model in 32 bits: latency
        dict(name="attn_3_h9_f32", op="attn", H=9, G=3, dim=64, batch=3, T=1, page=16, tokens=1100, longest=517,
             empty=0, inputs="f32", joined=False),
        # a ragged batch decoding, one token each
        dict(name="attn_64_h32_ragged", op="attn", H=32, G=8, dim=128, batch=64, T=1, page=16, tokens=200000,
             longest=8191, empty=1, inputs="bf16", joined=True),
        # one request with a long document, few heads: the work has to be split along the cache
        dict(name="attn_1x131k_h16", op="attn", H=16, G=2, dim=128, batch=1, T=1, page=64, tokens=131072,
             longest=131072, empty=0, inputs="bf16", joined=False),
        # drafts of four tokens, verified
        dict(name="attn_32x4_h40", op="attn", H=40, G=8, dim=128, batch=32, T=4, page=32, tokens=80000, longest=6001,
             empty=0, inputs="bf16", joined=False),
        # a request forked: its last page, which is not full, for each of a few layers
        dict(name="copy_2x8", op="copy", pools=8, pages=9, n=2, page=16, G=2, dim=128, inputs="bf16", skipped=0),
        # a batch of forks over the keys and values of 48 layers
        dict(name="copy_64x96", op="copy", pools=96, pages=150, n=64, page=16, G=8, dim=128, inputs="bf16", skipped=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


CHANNELS = [5376, 10240, 18432, 512, 768, 1000, 333, 2304]
HEADS = [(32, 8), (40, 8), (16, 2), (16, 16), (9, 3), (14, 2), (20, 4), (64, 8), (8, 1)]


def _longest(rng, total, n):
    return total if n == 1 else min(total - n + 1, int(math.ceil(total / n * rng.uniform(1.0, 3.0))))


def draw(rng):
    op = rng.choice(["conv", "cstep", "rope", "attn", "attn", "attn", "copy"])
    inputs = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "cstep"):
        c = dict(op=op, C=rng.choice(CHANNELS), width=rng.choice([4, 4, 4, 3, 2]), inputs=inputs,
                 bias=rng.random() < 0.7, silu=rng.random() < 0.8, sliced=rng.random() < 0.5)
        if op == "conv":
            c["R"] = rng.choice([c["width"], 8, 11])
            c["tokens"] = _log(rng, 1, 8192 if inputs == "bf16" else 4096)
            c["seqs"] = min(c["tokens"], _log(rng, 1, 40))
            c.update(longest=_longest(rng, c["tokens"], c["seqs"]), initial=rng.random() < 0.6)
            return c
        c["T"] = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        c["R"] = c["width"] - 1 + c["T"] + rng.choice([0, 0, 1, 5])
        c["batch"] = _log(rng, 1, 256)
        c["pads"] = rng.choice([0, 0, 1]) if c["batch"] > 1 else 0
        return c
    H, G = rng.choice(HEADS)
    dim = rng.choice([128, 128, 64])
    if op == "rope":
        c = dict(op=op, H=H, G=G, dim=dim, rot=rng.choice([dim, dim, dim // 2, 24]), page=rng.choice([16, 64, 1, 7]),
                 far=_log(rng, 300, 1000000), inputs=inputs, swap=rng.random() < 0.4, sliced=rng.random() < 0.5,
                 joined=rng.random() < 0.5, amplitude=rng.choice([1.0, 1.0, 1.25]))
        if rng.random() < 0.5:
            c.update(packed=_log(rng, 1, 4096), T=0)
            c["batch"] = min(c["packed"], _log(rng, 1, 24))
            c["longest"] = _longest(rng, c["packed"], c["batch"])
        else:
            c.update(packed=0, longest=0, T=rng.choice([1, 1, 2, 4, 5]), batch=_log(rng, 1, 256))
        return c
    if op == "copy":
        c = dict(op=op, pools=_log(rng, 1, 96), n=_log(rng, 1, 48), page=rng.choice([16, 32, 7]), G=G, dim=dim,
                 inputs=inputs)
        c["pages"] = 2 * c["n"] + rng.randrange(1, 20)
        while c["pools"] * c["pages"] * c["page"] * G * dim * SIZE[inputs] > 4e8:
            c["pools"] = (c["pools"] + 1) // 2 if c["pools"] > 1 else 1
            c["n"] = max(1, c["n"] * 2 // 3)
            c["pages"] = 2 * c["n"] + 7
        c["skipped"] = rng.choice([0, 1]) if c["n"] > 1 else 0
        return c
    c = dict(op=op, H=H, G=G, dim=dim, batch=_log(rng, 1, 128), T=rng.choice([1, 1, 1, 1, 2, 3, 4, 8]),
             page=rng.choice([16, 16, 32, 64, 128, 1, 7]), inputs=inputs, joined=rng.random() < 0.5)
    most = min(200000 * 1024 // (G * dim * (2 if inputs == "f32" else 1)), 400000)
    c["tokens"] = max(c["batch"] * c["T"], _log(rng, 16, most))
    c["empty"] = rng.choice([0, 0, 1]) if c["batch"] > 2 else 0
    live = c["batch"] - c["empty"]
    c["longest"] = max(c["T"], _longest(rng, c["tokens"], live)) if live > 1 else c["tokens"]
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _lengths(S, total, top, seed):
    """Lengths of S sequences that come to `total`: the longest as stated, the others at random, all at least one."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    if S == 1:
        return [total]
    left = total - top
    w = torch.rand(S - 1, generator=g).double() ** 2 + 1e-3
    n = torch.clamp((w / w.sum() * left).floor().long(), 1, top).tolist()
    i = 0
    while sum(n) != left:  # hand out (or take back) the rest, within [1, longest]
        step = 1 if sum(n) < left else -1
        if 1 <= n[i % len(n)] + step <= top:
            n[i % len(n)] += step
        i += 1
    at = int(torch.randint(0, S, (1,), generator=g))
    return n[:at] + [top] + n[at:]


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rand(g, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _slots(seed, batch, pads):
    """Distinct slots 1 .. batch in random order (slot 0 is nobody's); `pads` of them are the pad slot."""
    g = torch.Generator().manual_seed(seed * 5 + 2)
    s = 1 + torch.randperm(batch, generator=g)
    if pads:
        s[torch.randperm(batch, generator=g)[:pads]] = -1
    return s.to(torch.int32).cuda()


def _pools(g, pages, page, G, dim, t, joined, fill):
    """The pages of one layer's keys and values, side by side in one tensor or in two."""
    make = (lambda *s: _randn(g, *s, dtype=t)) if fill else (lambda *s: torch.zeros(s, dtype=t, device="cuda"))
    if joined:
        kv = make(pages, 2, page, G, dim)
        return kv[:, 0], kv[:, 1]
    return make(pages, page, G, dim), make(pages, page, G, dim)


def _table(seed, first, last, page, width):
    """A page table: request b holds pages for the tokens first[b] .. last[b] - 1, scattered over the pool; entries
    that nothing needs are -1.  Returns it and a number of pages that holds them wherever the tokens begin."""
    g = torch.Generator().manual_seed(seed * 3 + 4)
    need = [(a // page, -(-b // page)) for a, b in zip(first, last)]
    count = sum(max(0, b - a) for a, b in need)
    free = (2 + torch.randperm(count, generator=g)).to(torch.int32)  # pages 0 and 1 are nobody's
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for r, (a, b) in enumerate(need):
        if b > a:
            table[r, a:b] = free[at:at + b - a]
            at += b - a
    return table.cuda(), 2 + sum((b - a) // page + 2 for a, b in zip(first, last))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TORCH[c["inputs"]]
    s = {"op": c["op"]}
    if c["op"] in ("conv", "cstep"):
        C, W = c["C"], c["width"]
        lead = (c["tokens"],) if c["op"] == "conv" else (c["batch"], c["T"])
        x = _randn(g, *lead, C + (C // 2 if c["sliced"] else 0), dtype=t)
        n = c["seqs"] if c["op"] == "conv" else c["batch"]
        s.update(x=x[..., -C:] if c["sliced"] else x, weight=_randn(g, C, W) / W ** 0.5,
                 bias=0.1 * _randn(g, C) if c["bias"] else None, silu=c["silu"],
                 cache=_randn(g, n + 1, c["R"], C, dtype=t))
        far = torch.randint(0, 100000, (n,), generator=g, device="cuda", dtype=torch.int32)
        if c["op"] == "conv":
            m = _lengths(n, c["tokens"], c["longest"], seed)
            s.update(cu=_i32([0] + m).cumsum(0, dtype=torch.int32), slots=_slots(seed, n, 0),
                     positions=far if c["initial"] else None)
        else:
            s.update(slots=_slots(seed, n, c["pads"]), positions=far)
        return s
    if c["op"] == "copy":
        # every layer's keys and values, of one allocation
        store = torch.randn((c["pools"], c["pages"], c["page"], c["G"], c["dim"]), generator=g, device="cuda", dtype=t)
        pools = list(store)
        h = torch.Generator().manual_seed(seed * 3 + 5)
        order = 1 + torch.randperm(c["pages"] - 1, generator=h)  # page 0 is nobody's
        src, dst = order[torch.randint(c["n"], c["pages"] - 1, (c["n"],), generator=h)], order[:c["n"]]
        skip = torch.randperm(c["n"], generator=h)[:c["skipped"]]
        src[skip], dst[skip] = -1, -1
        s.update(store=store, pools=pools, src=src.to(torch.int32).cuda(), dst=dst.to(torch.int32).cuda(),
                 elements=c["page"] * c["G"] * c["dim"])  # of a page
        if own:
            import mamba_replayssm_state_gb300 as rsm
            s.update(ptrs=rsm.pointer_table(pools), strides=rsm.stride_table(pools))
        return s
    H, G, dim, b = c["H"], c["G"], c["dim"], c["batch"]
    if c["op"] == "rope":
        n = _lengths(b, c["packed"], c["longest"], seed) if c["packed"] else [c["T"]] * b
        h = torch.Generator().manual_seed(seed * 11 + 6)
        first = torch.randint(0, c["far"], (b,), generator=h).tolist()
        lengths = [f + m for f, m in zip(first, n)]
        table, pages = _table(seed, first, lengths, c["page"], -(-max(lengths) // c["page"]) + 1)
        lead = (c["packed"],) if c["packed"] else (b, c["T"])
        if c["sliced"]:
            q, k, v = _randn(g, *lead, (H + 2 * G) * dim, dtype=t).split([H * dim, G * dim, G * dim], dim=-1)
            q, k, v = q.unflatten(-1, (H, dim)), k.unflatten(-1, (G, dim)), v.unflatten(-1, (G, dim))
        else:
            q, k, v = (_randn(g, *lead, m, dim, dtype=t) for m in (H, G, G))
        k_cache, v_cache = _pools(g, pages, c["page"], G, dim, t, c["joined"], False)
        s.update(q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, table=table, lengths=_i32(lengths),
                 freq=(500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda(),
                 cu=_i32([0] + n).cumsum(0, dtype=torch.int32) if c["packed"] else None,
                 swap=c["swap"], amplitude=c["amplitude"])
        return s
    live = b - c["empty"]
    n = _lengths(live, c["tokens"], c["longest"], seed)
    n = [max(m, c["T"]) for m in n] + [0] * c["empty"]
    table, pages = _table(seed, [0] * b, n, c["page"], -(-max(n) // c["page"]) + 2)
    k_cache, v_cache = _pools(g, pages, c["page"], G, dim, t, c["joined"], True)
    s.update(q=2.0 * _randn(g, b, c["T"], H, dim, dtype=t), k_cache=k_cache, v_cache=v_cache, table=table,
             lengths=_i32(n), host_lengths=n)  # the scheduler that admitted the requests knows them
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"conv": _conv, "cstep": _cstep, "rope": _rope, "attn": _attn, "copy": _copy}[s["op"]](s)


def _run_own(s):
    import mamba_replayssm_state_gb300 as rsm
    if s["op"] == "conv":
        y = rsm.causal_conv(s["x"], s["weight"], s["cu"], s["bias"], s["cache"], s["slots"], s["positions"],
                            silu=s["silu"])
        return {"y": y, "cache": s["cache"]}
    if s["op"] == "cstep":
        y = rsm.causal_conv_step(s["x"], s["weight"], s["cache"], s["slots"], s["positions"], s["bias"], silu=s["silu"])
        return {"y": y, "cache": s["cache"]}
    if s["op"] == "rope":
        q = rsm.rotary_append(s["q"], s["k"], s["v"], s["freq"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                              s["cu"], interleaved=s["swap"], amplitude=s["amplitude"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "attn":
        return {"y": rsm.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"])}
    rsm.copy_pages(s["ptrs"], s["strides"], s["src"], s["dst"], dtype=s["store"].dtype, page_elements=s["elements"],
                   num_pages=s["store"].shape[1])
    return {"pools": s["store"]}


def _silu(v):
    return v / (1.0 + (-v).exp())


def _conv(s):
    x, cu, cache = s["x"].float(), s["cu"].long(), s["cache"]
    W, R = s["weight"].shape[1], cache.shape[1]
    slots, n = s["slots"].long(), cu[1:] - cu[:-1]
    at = torch.arange(x.shape[0], device="cuda")
    owner = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    inside = at - cu[owner]                                       # a token's place in its sequence
    y = x * s["weight"][:, W - 1]
    for j in range(1, min(W, x.shape[0] + 1)):
        before = torch.where((inside >= j)[:, None], x.roll(j, 0), 0.0)
        y += before * s["weight"][:, W - 1 - j]
    if s["positions"] is not None:                                # inputs of earlier calls, for the first tokens
        p = s["positions"].long()
        for j in range(1, W):
            old = torch.where((p >= j)[:, None], cache[slots, (p - j) % R].float(), 0.0)
            for i in range(W - j):
                live = (n > i)[:, None]
                y.index_add_(0, torch.where(n > i, cu[:-1] + i, 0), torch.where(live, old * s["weight"][:, W - 1 - j - i], 0.0))
    else:
        p = torch.zeros_like(n)
    if s["bias"] is not None:
        y += s["bias"]
    if s["silu"]:
        y = _silu(y)
    rows = []
    for j in range(1, W):
        row = (p + n - j) % R
        rows.append((row, torch.where((n >= j)[:, None], s["x"][(cu[1:] - j).clamp(min=0)], cache[slots, row])))
    for row, v in rows:
        cache[slots, row] = v
    return {"y": y.to(s["x"].dtype), "cache": cache}


def _cstep(s):
    x, cache = s["x"].float(), s["cache"]
    W, R, T = s["weight"].shape[1], cache.shape[1], x.shape[1]
    live, slots, p = s["slots"] >= 0, s["slots"].clamp(min=0).long(), s["positions"].long()
    back = torch.arange(W - 1, 0, -1, device="cuda")
    old = cache[slots[:, None], (p[:, None] - back) % R].float()
    old = torch.where((p[:, None] >= back)[..., None], old, 0.0)
    every = torch.cat([old, x], 1)
    y = sum(every[:, j:j + T] * s["weight"][:, j] for j in range(W))
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["silu"]:
        y = _silu(y)
    row = (p[:, None] + torch.arange(T, device="cuda")) % R
    cache[slots[:, None], row] = torch.where(live[:, None, None], s["x"], cache[slots[:, None], row])
    return {"y": torch.where(live[:, None, None], y, 0.0).to(s["x"].dtype), "cache": cache}


def _rotate(v, cos, sin, swap):
    """v [tokens, heads, dim] by angles [tokens, pairs]; swap: pairs are neighbours, else halves."""
    half = cos.shape[-1]
    a, b = (v[..., 0:2 * half:2], v[..., 1:2 * half:2]) if swap else (v[..., :half], v[..., half:2 * half])
    c, d = cos[:, None], sin[:, None]
    x, y = a * c - b * d, b * c + a * d
    turned = torch.stack([x, y], -1).flatten(-2) if swap else torch.cat([x, y], -1)
    return torch.cat([turned, v[..., 2 * half:]], -1)


def _rope(s):
    q, k, v = (s[n].float() if s["cu"] is not None else s[n].float().flatten(0, 1) for n in ("q", "k", "v"))
    if s["cu"] is not None:
        cu = s["cu"].long()
        at = torch.arange(q.shape[0], device="cuda")
        owner = torch.searchsorted(cu[1:].contiguous(), at, right=True)
        p = s["lengths"].long()[owner] - cu[owner + 1] + at
    else:
        b, T = s["q"].shape[:2]
        owner = torch.arange(b, device="cuda").repeat_interleave(T)
        p = (s["lengths"].long()[:, None] - T + torch.arange(T, device="cuda")).flatten()
    angle = p.double()[:, None] * s["freq"].double()
    cos, sin = angle.cos().float() * s["amplitude"], angle.sin().float() * s["amplitude"]
    page = s["k_cache"].shape[1]
    to = s["table"].long()[owner, p // page], p % page
    s["k_cache"][to] = _rotate(k, cos, sin, s["swap"]).to(s["k"].dtype)
    s["v_cache"][to] = v.to(s["v"].dtype)
    out = _rotate(q, cos, sin, s["swap"]).to(s["q"].dtype)
    return {"q": out.view(s["q"].shape), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn(s):
    q = s["q"]
    T, H, dim = q.shape[1:]
    page, G = s["k_cache"].shape[1:3]
    out = torch.zeros_like(q)
    for b, n in enumerate(s["host_lengths"]):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:n].float().permute(1, 2, 0)     # [G, dim, n]
        v = s["v_cache"][pages].flatten(0, 1)[:n].float().transpose(0, 1)      # [G, n, dim]
        qb = q[b].float().unflatten(1, (G, -1)).permute(1, 0, 2, 3)            # [G, T, H / G, dim]
        w = (qb.flatten(1, 2) @ k).unflatten(1, (T, -1)) * dim ** -0.5
        if T > 1:
            last = n - T + torch.arange(T, device="cuda")
            w = torch.where(torch.arange(n, device="cuda") <= last[:, None, None], w, -math.inf)
        w = (w - w.amax(-1, keepdim=True)).exp()
        y = (w.flatten(1, 2) @ v).unflatten(1, (T, -1)) / w.sum(-1, keepdim=True)
        out[b] = y.permute(1, 0, 2, 3).flatten(1, 2).to(q.dtype)
    return {"y": out}


def _copy(s):
    src, dst = s["src"].clamp(min=0).long(), s["dst"].clamp(min=0).long()  # a skipped pair: page 0 over itself
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return {"pools": s["store"]}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c, e = case, SIZE[case["inputs"]]
    if c["op"] == "conv":
        n, W = c["tokens"] * c["C"], c["width"]
        rows = c["seqs"] * (W - 1) * c["C"] * (2 if c["initial"] else 1)
        return {"bytes": e * (2 * n + rows) + 4 * c["C"] * (W + 1), "flops": n * (2 * W + (4 if c["silu"] else 0))}
    if c["op"] == "cstep":
        W, b = c["width"], c["batch"] - c["pads"]
        n = b * c["T"] * c["C"]
        return {"bytes": e * (3 * n + b * (W - 1) * c["C"]) + 4 * c["C"] * (W + 1),
                "flops": n * (2 * W + (4 if c["silu"] else 0))}
    if c["op"] == "copy":
        n = (c["n"] - c["skipped"]) * c["pools"] * c["page"] * c["G"] * c["dim"]
        return {"bytes": 2 * e * n, "flops": 0}
    H, G, dim = c["H"], c["G"], c["dim"]
    if c["op"] == "rope":
        n = c["packed"] or c["batch"] * c["T"]
        return {"bytes": 2 * e * n * (H + 2 * G) * dim + 2 * c["rot"], "flops": 3 * n * (H + G) * c["rot"]}
    live = c["batch"] - c["empty"]
    seen = max(c["tokens"], live * c["T"])
    return {"bytes": 2 * e * seen * G * dim + 2 * e * c["batch"] * c["T"] * H * dim,
            "flops": 4 * seen * c["T"] * H * dim}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"conv": _exact_conv, "cstep": _exact_conv, "rope": _exact_rope, "attn": _exact_attn,
            "copy": _exact_copy}[c["op"]](s)


def _exact_conv(s):
    """A request after the other: its earlier inputs and its own in one row of tokens, windows of it weighed."""
    x, cache, W = s["x"], s["cache"].double(), s["weight"].shape[1]
    R = cache.shape[1]
    slots = s["slots"].tolist()
    first = [0] * len(slots) if s["positions"] is None else s["positions"].tolist()
    if s["op"] == "conv":
        cu = s["cu"].tolist()
        spans = [x[a:b] for a, b in zip(cu, cu[1:])]
    else:
        spans = list(x)
    out = []
    for slot, p, own_x in zip(slots, first, spans):
        if slot < 0:
            out.append(torch.zeros(own_x.shape, dtype=torch.float64, device="cuda"))
            continue
        own_x = own_x.double()
        past = [cache[slot, (p - j) % R].clone() if p >= j else torch.zeros_like(own_x[0]) for j in range(W - 1, 0, -1)]
        line = torch.cat([torch.stack(past), own_x]) if past else own_x
        y = torch.zeros_like(own_x) if s["bias"] is None else s["bias"].double().expand_as(own_x).clone()
        for j in range(W):
            y += line[j:j + len(own_x)] * s["weight"][:, j].double()
        out.append(y * torch.sigmoid(y) if s["silu"] else y)
        kept = len(own_x) if s["op"] == "cstep" else min(len(own_x), W - 1)
        for i in range(len(own_x) - kept, len(own_x)):
            cache[slot, (p + i) % R] = own_x[i]
    return {"y": torch.cat(out) if s["op"] == "conv" else torch.stack(out), "cache": cache}


def _exact_rope(s):
    """Pairs as complex numbers, turned by e^(i p f)."""
    page, half = s["k_cache"].shape[1], s["freq"].numel()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    lengths, table = s["lengths"].tolist(), s["table"]
    cu = None if s["cu"] is None else s["cu"].tolist()
    out = []

    def turn(v, p):
        v = v.double()
        part = v[..., :2 * half]
        pair = part.unflatten(-1, (half, 2)) if s["swap"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_complex(pair.contiguous())
        z = z * torch.polar(torch.full((len(p), 1, half), float(s["amplitude"]), dtype=torch.float64, device="cuda"),
                            (p[:, None] * s["freq"].double())[:, None])
        z = torch.view_as_real(z)
        z = z if s["swap"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), v[..., 2 * half:]], -1)

    for b, n in enumerate(lengths):
        rows = slice(cu[b], cu[b + 1]) if cu else b
        q, k, v = s["q"][rows], s["k"][rows], s["v"][rows]
        at = torch.arange(n - len(q), n, device="cuda")
        out.append(turn(q, at.double()))
        to = table[b, at // page].long(), at % page
        kc[to], vc[to] = turn(k, at.double()), v.double()
    return {"q": torch.cat(out) if cu else torch.stack(out), "k_cache": kc, "v_cache": vc}


def _exact_attn(s):
    """Request by request and group by group: logarithms of the sums of exponentials, then the weighted values."""
    q = s["q"]
    T, H, dim = q.shape[1:]
    page, G = s["k_cache"].shape[1:3]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        rows = s["table"][b, at // page].long(), at % page
        hidden = at > n - T + torch.arange(T, device="cuda")[:, None]
        for j in range(G):
            k, v = s["k_cache"][:, :, j][rows].double(), s["v_cache"][:, :, j][rows].double()
            h = slice(j * (H // G), (j + 1) * (H // G))
            w = torch.einsum("thd,nd->htn", q[b, :, h].double(), k) / math.sqrt(dim)
            w = w.masked_fill(hidden, -math.inf)
            w = torch.exp(w - torch.logsumexp(w, -1, keepdim=True))
            out[b, :, h] = torch.einsum("htn,nd->thd", w, v)
    return {"y": out}


def _exact_copy(s):
    new, old = s["store"].double(), s["store"]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        if a >= 0:
            new[:, b] = old[:, a]
    return {"pools": new}
