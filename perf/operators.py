"""Cases of the block operators: the linear-attention layer of a Mamba-2 style
model from prompt to decoded token, and the norms around it.

  prefill   ssm_prefill        packed prompts -> outputs and state slots (chunked form)
  step      ssm_step           new tokens of running requests, state slot -> state slot (recurrent form)
  decode    replayssm_decode   new tokens from a checkpoint slot plus its replay ring, the state only read
  add_norm  add_rms_norm       residual + scale * x, then RMS norm (before a block)
  gate_norm gated_rms_norm     x * silu(z), then RMS norm over groups (after the block)

Head counts, groups, state sizes and rings are those of the package's own
workloads (80 heads in one group with fp32 state; 128 heads in groups of 16
with fp16 state; 256 heads in groups of 32 with bf16 or one-byte state; 64 x
128 states; rings of 8, 16 and 64 rows).
"""
import math

import torch

own = False

EPS = 1e-5
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8,
         "fp8": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1, "fp8": 1}


def listed():
    return [
        # one short prompt alone: a first token's latency
        dict(name="prefill_1x37_h80", op="prefill", H=80, G=1, dim=64, dstate=128, seqs=1, tokens=37, longest=37,
             inputs="bf16", state="f32", initial=False, skip=True, packed=True),
        # a ragged batch of prompts, from one token to a couple of thousand
        dict(name="prefill_16seq_8k_h128", op="prefill", H=128, G=8, dim=64, dstate=128, seqs=16, tokens=8192,
             longest=2011, inputs="bf16", state="f16", initial=False, skip=True, packed=False),
        # the next pieces of four long prompts: states come from earlier pieces
        dict(name="prefill_4seq_8k_h256", op="prefill", H=256, G=8, dim=64, dstate=128, seqs=4, tokens=8192,
             longest=2560, inputs="bf16", state="bf16", initial=True, skip=True, packed=True),
        # one long document: few heads, so the work has to be split along the sequence
        dict(name="prefill_1x32k_h80", op="prefill", H=80, G=1, dim=64, dstate=128, seqs=1, tokens=32768,
             longest=32768, inputs="bf16", state="f32", initial=False, skip=True, packed=True),
        # one request decoding alone
        dict(name="step_1_h80", op="step", H=80, G=1, dim=64, dstate=128, batch=1, T=1, inputs="bf16", state="f32",
             pads=0, skip=True),
        # a full batch decoding, one token each
        dict(name="step_256_h256", op="step", H=256, G=8, dim=64, dstate=128, batch=256, T=1, inputs="bf16",
             state="bf16", pads=0, skip=True),
        # a full batch decoding from checkpoints and rings: the state is only read
        dict(name="decode_256_h256", op="decode", H=256, G=8, dim=64, dstate=128, batch=256, T=1, R=8, inputs="bf16",
             state="bf16", pads=3, skip=True),
        # verification of drafts of four tokens, one-byte states
        dict(name="decode_64x4_h256_i8", op="decode", H=256, G=8, dim=64, dstate=128, batch=64, T=4, R=16,
             inputs="bf16", state="i8", pads=0, skip=True),
        # the norm before a block for one token
        dict(name="add_norm_1x5120", op="add_norm", rows=1, dim=5120, inputs="bf16", residual="f32"),
        # the same for a prompt's tokens, residual stream in 32 bits
        dict(name="add_norm_8192x4096", op="add_norm", rows=8192, dim=4096, inputs="bf16", residual="f32"),
        # the gated norm after the layer for a decoding batch
        dict(name="gate_norm_64x8192", op="gate_norm", rows=64, dim=8192, group=1024, inputs="bf16", first=False,
             packed=True),
        # the same for a prompt's tokens
        dict(name="gate_norm_8192x16384", op="gate_norm", rows=8192, dim=16384, group=2048, inputs="bf16",
             first=False, packed=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    H, G = rng.choice([(80, 1), (128, 8), (256, 8), (24, 1), (48, 2), (20, 4), (6, 2), (9, 3), (32, 32)])
    return dict(H=H, G=G)


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "decode", "add_norm", "gate_norm"])
    if op == "prefill":
        c = dict(op=op, **_heads(rng), dim=64, dstate=128)
        c["tokens"] = _log(rng, 1, max(1, min(16384, 32768 * 80 // c["H"] // 2)))
        c["seqs"] = min(c["tokens"], _log(rng, 1, 24))
        c["inputs"] = "bf16"
        if rng.random() < 0.2:  # the small forms: other state sizes, inputs in 32 bits
            c["tokens"] = min(c["tokens"], rng.randrange(300, 700))
            c["seqs"] = min(c["tokens"], c["seqs"])
            c["dim"], c["dstate"] = rng.choice([(16, 16), (64, 64), (64, 128)])
            c["inputs"] = rng.choice(["f32", "bf16"])
        mean = c["tokens"] / c["seqs"]
        c["longest"] = c["tokens"] if c["seqs"] == 1 else min(c["tokens"] - c["seqs"] + 1,
                                                               int(math.ceil(mean * rng.uniform(1.0, 3.0))))
        c.update(state=rng.choice(["f32", "bf16", "f16"]), initial=rng.random() < 0.5, skip=rng.random() < 0.7,
                 packed=rng.random() < 0.5)
        return c
    if op in ("step", "decode"):
        c = dict(op=op, **_heads(rng), dim=64, dstate=128, batch=_log(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 3, 4, 8]))
        c["inputs"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c["state"] = rng.choice(["f32", "bf16", "f16"] if op == "step" else ["f32", "bf16", "f16", "i8", "fp8"])
        if c["state"] == "f32":
            c["batch"] = min(c["batch"], 128)
        if op == "decode":
            c["R"] = rng.choice([8, 16, 16, 64])
        c.update(pads=rng.choice([0, 0, 1]) if c["batch"] > 1 else 0, skip=rng.random() < 0.7)
        return c
    rows = _log(rng, 1, 8192)
    if op == "add_norm":
        return dict(op=op, rows=rows, dim=rng.choice([1024, 2048, 4096, 5120, 8192, 1000 + rng.randrange(1, 500)]),
                    inputs=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["f32", "bf16"]))
    group, n = rng.choice([(512, 8), (1024, 8), (2048, 8), (5120, 1), (4096, 1), (64, 80), (200, 5)])
    return dict(op=op, rows=rows, dim=group * n, group=group, inputs=rng.choice(["bf16", "bf16", "f32"]),
                first=rng.random() < 0.3, packed=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _lengths(case, seed):
    """Host lengths of the packed sequences: the longest as stated, the others at random, all at least one token."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    S, T, top = case["seqs"], case["tokens"], case["longest"]
    if S == 1:
        return [T]
    left = T - top
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rand(g, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _split(g, lead, H, G, dim, dstate, dtype, packed):
    """x, B and C of the new tokens: one projection's slices where packed, tensors of their own otherwise."""
    if packed:
        xbc = _randn(g, *lead, H * dim + 2 * G * dstate, dtype=dtype)
        x, B, C = xbc.split([H * dim, G * dstate, G * dstate], dim=-1)
        return x.unflatten(-1, (H, dim)), B.unflatten(-1, (G, dstate)), C.unflatten(-1, (G, dstate))
    return (_randn(g, *lead, H, dim, dtype=dtype), _randn(g, *lead, G, dstate, dtype=dtype),
            _randn(g, *lead, G, dstate, dtype=dtype))


def _pool(g, slots, H, dim, dstate, kind):
    """A state pool and, for one-byte states, its scale per row."""
    if kind in ("i8", "fp8"):
        v = torch.randint(-127, 128, (slots, H, dim, dstate), generator=g, device="cuda", dtype=torch.int8)
        if kind == "fp8":
            v = (v.to(torch.float16) * 3.5).to(torch.float8_e4m3fn)
        return v, _rand(g, 0.5, 2.0, slots, H, dim) * (4.0 / (127.0 if kind == "i8" else 448.0))
    return torch.randn((slots, H, dim, dstate), generator=g, device="cuda", dtype=TORCH[kind]), None


def _rows(pool, slots):
    """The states of `slots` (a pad reads slot 0's) as values; one-byte codes are gathered as bytes."""
    at = slots.clamp(min=0).long()
    return pool.view(torch.uint8)[at].view(pool.dtype) if pool.element_size() == 1 else pool[at]


def _slots(seed, batch, pads, first):
    """Distinct slots first .. first + batch - 1 in random order; `pads` of them are the pad slot."""
    g = torch.Generator().manual_seed(seed * 5 + first)
    s = first + torch.randperm(batch, generator=g)
    if pads:
        s[torch.randperm(batch, generator=g)[:pads]] = -1
    return s.to(torch.int32).cuda()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"op": c["op"]}
    if c["op"] in ("add_norm", "gate_norm"):
        t = TORCH[c["inputs"]]
        s["weight"] = _rand(g, 0.5, 1.5, c["dim"])
        if c["op"] == "add_norm":
            s.update(x=_randn(g, c["rows"], c["dim"], dtype=t), scale=0.5,
                     residual=(3.0 * _randn(g, c["rows"], c["dim"])).to(TORCH[c["residual"]]))
        else:
            zx = _randn(g, c["rows"], 2 * c["dim"], dtype=t) if c["packed"] else None
            s.update(x=zx[:, c["dim"]:] if c["packed"] else _randn(g, c["rows"], c["dim"], dtype=t),
                     z=zx[:, :c["dim"]] if c["packed"] else _randn(g, c["rows"], c["dim"], dtype=t),
                     group=c["group"], first=c["first"])
        return s
    H, G, dim, dstate = c["H"], c["G"], c["dim"], c["dstate"]
    s["A"] = -_rand(g, 0.5, 2.0, H)
    s["D"] = _randn(g, H) if c["skip"] else None
    t = TORCH[c["inputs"]]
    if c["op"] == "prefill":
        n = _lengths(c, seed)
        s["cu"] = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        s["longest"] = max(n)  # the scheduler that packed the batch knows it
        s["x"], s["B"], s["C"] = _split(g, (c["tokens"],), H, G, dim, dstate, t, c["packed"])
        s["dt"] = _rand(g, 0.001, 0.1, c["tokens"], H)
        s["state"], _ = _pool(g, 2 * c["seqs"] + 1, H, dim, dstate, c["state"])
        s["initial"] = _slots(seed, c["seqs"], 0, 1) if c["initial"] else None
        s["final"] = _slots(seed, c["seqs"], 0, 1 + c["seqs"])
        return s
    b, T = c["batch"], c["T"]
    s["x"], s["B"], s["C"] = _split(g, (b, T), H, G, dim, dstate, t, False)
    s["dt"] = _rand(g, 0.001, 0.1, b, T, H)
    # slot 0 is nobody's
    if c["op"] == "step":
        s["state"], _ = _pool(g, 2 * b + 1, H, dim, dstate, c["state"])
        s["src"] = _slots(seed, b, c["pads"], 1)
        s["dst"] = torch.where(s["src"] < 0, s["src"], _slots(seed, b, 0, 1 + b))
        return s
    s["state"], s["scale"] = _pool(g, b + 1, H, dim, dstate, c["state"])
    s["src"] = _slots(seed, b, c["pads"], 1)
    R = c["R"]
    s["x_cache"], s["B_cache"] = _randn(g, b + 1, R, H, dim, dtype=t), _randn(g, b + 1, R, G, dstate, dtype=t)
    s["dt_cache"] = _rand(g, 0.001, 0.1, b + 1, R, H)
    s["ring_start"] = torch.randint(0, R, (b,), generator=g, device="cuda", dtype=torch.int32)
    s["ring_len"] = torch.randint(0, R - T + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _prefill, "step": _step, "decode": _decode, "add_norm": _add_norm,
            "gate_norm": _gate_norm}[s["op"]](s)


def _run_own(s):
    import mamba_replayssm_state_gb300 as rsm
    if s["op"] == "prefill":
        y = rsm.ssm_prefill(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["state"], initial_slots=s["initial"],
                            final_slots=s["final"], D=s["D"])
        return {"y": y, "state": s["state"]}
    if s["op"] == "step":
        y = rsm.ssm_step(s["state"], s["src"], s["x"], s["dt"], s["A"], s["B"], s["C"], dst_slots=s["dst"], D=s["D"])
        return {"y": y, "state": s["state"]}
    if s["op"] == "decode":
        y = rsm.replayssm_decode(s["state"], s["src"], s["x_cache"], s["B_cache"], s["dt_cache"], s["ring_start"],
                                 s["ring_len"], s["x"], s["dt"], s["A"], s["B"], s["C"], state_scale=s["scale"],
                                 D=s["D"])
        return {"y": y, "x_cache": s["x_cache"], "B_cache": s["B_cache"], "dt_cache": s["dt_cache"]}
    if s["op"] == "add_norm":
        y, r = rsm.add_rms_norm(s["x"], s["residual"], s["weight"], residual_scale=s["scale"], eps=EPS)
        return {"y": y, "residual": r}
    return {"y": rsm.gated_rms_norm(s["x"], s["z"], s["weight"], group_size=s["group"], eps=EPS,
                                    norm_before_gate=s["first"])}


def _sums(a):
    """[..., n] -> [..., n, n]: the sum of a over (j, i], -inf where j > i, each added up from its own terms."""
    n = a.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=a.device).tril(-1)
    m = torch.where(low, a[..., :, None], 0.0).cumsum(-2)
    return torch.where(low.logical_not().triu(1), -math.inf, m)


def _store(pool, slots, values):
    """values -> pool[slots] where the slot is one; a pad writes slot 0 (nobody's) back over itself."""
    at = slots.clamp(min=0).long()
    live = (slots >= 0).view(-1, *[1] * (values.dim() - 1))
    pool[at] = torch.where(live, values.to(pool.dtype), pool[at])


def _heads_of(v, H):
    """Group tensors [..., G, n] for every head: [..., H, n]."""
    return v.float().repeat_interleave(H // v.shape[-2], dim=-2)


def _prefill(s):
    Q = 64
    x, dt, A, cu = s["x"], s["dt"], s["A"], s["cu"]
    S, H, dim = cu.numel() - 1, x.shape[1], x.shape[2]
    G, dstate = s["B"].shape[1:]
    nc = -(-s["longest"] // Q)
    t = torch.arange(nc * Q, device="cuda")
    live = t < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(live, cu[:-1, None] + t, 0).long()
    pick = lambda v: torch.where(live.view(S, -1, *[1] * (v.dim() - 1)), v.float()[at], 0.0).unflatten(1, (nc, Q))  # noqa: E731
    xs, Bs, Cs, dts = pick(x), pick(s["B"]), pick(s["C"]), pick(dt)  # [S, nc, Q, ...]
    a = (dts * A).transpose(2, 3)                                    # [S, nc, H, Q]
    xd = (xs * dts[..., None]).transpose(2, 3)                       # [S, nc, H, Q, dim]
    Bg, Cg = Bs.transpose(2, 3), Cs.transpose(2, 3)                  # [S, nc, G, Q, dstate]
    per = H // G
    dots = (Cg @ Bg.transpose(-1, -2)).repeat_interleave(per, dim=2)
    y = (dots * _sums(a).exp()) @ xd
    total = a.sum(-1)                                                # [S, nc, H]
    after = a.flip(-1).cumsum(-1).flip(-1) - a                       # the decay of a token to its chunk's end
    add = (xd * after.exp()[..., None]).transpose(-1, -2).unflatten(2, (G, per)) @ Bg[:, :, :, None]
    first = torch.zeros(S, 1, H, dim, dstate, device="cuda") if s["initial"] is None else \
        s["state"][s["initial"].long()].float()[:, None]
    add = torch.cat([first, add.flatten(2, 3)], 1)                   # [S, nc + 1, H, dim, dstate]
    steps = torch.nn.functional.pad(total, (0, 0, 1, 0)).permute(0, 2, 1)  # [S, H, nc + 1]
    states = _sums(steps).exp() @ add.transpose(1, 2).flatten(3)     # [S, H, nc + 1, dim * dstate]
    states = states.unflatten(-1, (dim, dstate)).transpose(1, 2)
    before = a.cumsum(-1).exp()[..., None]
    y = y + before * (Cg[:, :, :, None] @ states[:, :-1].unflatten(2, (G, per)).transpose(-1, -2)).flatten(2, 3)
    y = y.transpose(2, 3)
    if s["D"] is not None:
        y = y + s["D"][:, None] * xs
    owner = torch.searchsorted(cu[1:].contiguous(), torch.arange(x.shape[0], device="cuda", dtype=torch.int32),
                               right=True)
    y = y.flatten(1, 2)[owner, torch.arange(x.shape[0], device="cuda") - cu[owner]]
    _store(s["state"], s["final"], states[:, -1])
    return {"y": y.to(x.dtype), "state": s["state"]}


def _tokens(a, dt, x, B, C, H):
    """Outputs of tokens from the tokens at and before them, and what each leaves in the state at the end:
    a, dt [b, n, H], x [b, n, H, dim], B [b, n, G, dstate], C [b, T, G, dstate] of the last T tokens."""
    T = C.shape[1]
    decay = _sums(a.transpose(1, 2)).exp()                                     # [b, H, n, n]
    dots = (C.float().transpose(1, 2) @ B.float().permute(0, 2, 3, 1)).repeat_interleave(H // C.shape[2], dim=1)
    p = dots * decay[:, :, -T:] * dt.transpose(1, 2)[:, :, None]               # [b, H, T, n]
    y = (p @ x.transpose(1, 2)).transpose(1, 2)
    left = decay[:, :, -1] * dt.transpose(1, 2)                                # [b, H, n]
    return y, left


def _step(s):
    x, dt = s["x"].float(), s["dt"]
    H = x.shape[2]
    a = dt * s["A"]
    old = _rows(s["state"], s["src"]).float()                     # [b, H, dim, dstate]
    y, left = _tokens(a, dt, x, s["B"], s["C"], H)
    C = _heads_of(s["C"], H).transpose(1, 2)                                   # [b, H, T, dstate]
    y = y + (a.cumsum(1).transpose(1, 2).exp()[..., None] * (C @ old.transpose(-1, -2))).transpose(1, 2)
    if s["D"] is not None:
        y = y + s["D"][:, None] * x
    B = _heads_of(s["B"], H).transpose(1, 2)
    new = a.sum(1).exp()[..., None, None] * old + (left[..., None] * x.transpose(1, 2)).transpose(-1, -2) @ B
    _store(s["state"], s["dst"], new)
    y = torch.where((s["src"] >= 0).view(-1, 1, 1, 1), y, 0.0)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _decode(s):
    H, T, R = s["x"].shape[2], s["x"].shape[1], s["x_cache"].shape[1]
    slot = s["src"].clamp(min=0).long()
    old = _rows(s["state"], s["src"]).float()
    if s["scale"] is not None:
        old = old * s["scale"][slot][..., None]
    i = torch.arange(R, device="cuda")
    row = (s["ring_start"][:, None] + i) % R                                   # [b, R], oldest first
    have = i < s["ring_len"][:, None]
    take = lambda v: torch.where(have.view(-1, R, *[1] * (v.dim() - 2)), v[slot[:, None], row].float(), 0.0)  # noqa: E731
    x = torch.cat([take(s["x_cache"]), s["x"].float()], 1)
    B = torch.cat([take(s["B_cache"]), s["B"].float()], 1)
    dt = torch.cat([take(s["dt_cache"]), s["dt"]], 1)
    a = dt * s["A"]                                                            # rows past ring_len decay by exp(0)
    y, _ = _tokens(a, dt, x, B, s["C"], H)
    C = _heads_of(s["C"], H).transpose(1, 2)
    y = y + (a.cumsum(1)[:, -T:].transpose(1, 2).exp()[..., None] * (C @ old.transpose(-1, -2))).transpose(1, 2)
    if s["D"] is not None:
        y = y + s["D"][:, None] * s["x"].float()
    live = s["src"] >= 0
    at = (s["ring_start"][:, None] + s["ring_len"][:, None] + torch.arange(T, device="cuda")) % R
    for cache, new in (("x_cache", s["x"]), ("B_cache", s["B"]), ("dt_cache", s["dt"])):
        v = s[cache]
        v[slot[:, None], at] = torch.where(live.view(-1, *[1] * (v.dim() - 1)), new, v[slot[:, None], at])
    y = torch.where(live.view(-1, 1, 1, 1), y, 0.0)
    return {"y": y.to(s["x"].dtype), "x_cache": s["x_cache"], "B_cache": s["B_cache"], "dt_cache": s["dt_cache"]}


def _rms(v, weight, group):
    w = v.unflatten(-1, (-1, group))
    return (w * torch.rsqrt(w.square().mean(-1, keepdim=True) + EPS)).flatten(-2) * weight


def _add_norm(s):
    r = s["residual"].float() + s["scale"] * s["x"].float()
    return {"y": _rms(r, s["weight"], r.shape[-1]).to(s["x"].dtype), "residual": r.to(s["residual"].dtype)}


def _gate_norm(s):
    x, z = s["x"].float(), s["z"].float()
    gate = z / (1.0 + (-z).exp())
    y = _rms(x, s["weight"], s["group"]) * gate if s["first"] else _rms(x * gate, s["weight"], s["group"])
    return {"y": y.to(s["x"].dtype)}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c, e = case, SIZE[case["inputs"]]
    if c["op"] == "add_norm":
        n = c["rows"] * c["dim"]
        return {"bytes": n * (2 * e + 2 * SIZE[c["residual"]]) + 4 * c["dim"], "flops": 6 * n}
    if c["op"] == "gate_norm":
        n = c["rows"] * c["dim"]
        return {"bytes": 3 * e * n + 4 * c["dim"], "flops": 10 * n}
    H, G, dim, dstate, st = c["H"], c["G"], c["dim"], c["dstate"], SIZE[c["state"]]
    tile = H * dim * dstate
    if c["op"] == "prefill":
        per = 2 * e * H * dim + 2 * e * G * dstate + 4 * H
        return {"bytes": c["tokens"] * per + c["seqs"] * tile * st * (2 if c["initial"] else 1),
                "flops": 4 * c["tokens"] * tile}
    b, T = c["batch"] - c["pads"], c["T"]
    per = 2 * e * H * dim + 2 * e * G * dstate + 4 * H                          # x in, y out, B, C, dt
    if c["op"] == "step":
        return {"bytes": b * (T * per + 2 * tile * st), "flops": 4 * b * T * tile}
    ring = e * H * dim + e * G * dstate + 4 * H                                # a ring row of x, B, dt
    mean = (c["R"] - T) / 2
    scales = 4 * H * dim if st == 1 else 0
    return {"bytes": b * (T * (per + ring) + mean * ring + tile * st + scales), "flops": 2 * b * T * tile}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda v: v.double()  # noqa: E731
    if s["op"] == "add_norm":
        r = f(s["residual"]) + s["scale"] * f(s["x"])
        return {"y": r / (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * f(s["weight"]), "residual": r}
    if s["op"] == "gate_norm":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, case["dim"], s["group"]):
            k = slice(i, i + s["group"])
            v, gate = f(s["x"][:, k]), f(s["z"][:, k]) * torch.sigmoid(f(s["z"][:, k]))
            v = v if s["first"] else v * gate
            v = v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * f(s["weight"][k])
            out[:, k] = v * gate if s["first"] else v
        return {"y": out}
    A, D = f(s["A"]), 0.0 if s["D"] is None else f(s["D"])[:, None]
    per = case["H"] // case["G"]

    def token(S, x, dt, B, C):
        """One step of the recurrence for a batch: S [b, H, dim, dstate] in place, the outputs returned."""
        S.mul_(torch.exp(dt * A)[..., None, None])
        Bh = B.repeat_interleave(per, 1)
        S.add_((dt[..., None] * x)[..., None] * Bh[:, :, None])
        if C is None:
            return None
        return torch.matmul(S, C.repeat_interleave(per, 1)[..., None])[..., 0] + D * x

    if s["op"] == "prefill":
        cu = s["cu"].tolist()
        n = [b - a for a, b in zip(cu, cu[1:])]
        order = sorted(range(len(n)), key=lambda k: -n[k])  # longest first: the live ones are a prefix
        start = torch.tensor([cu[k] for k in order], device="cuda")
        final = torch.empty(len(n), case["H"], case["dim"], case["dstate"], dtype=torch.float64, device="cuda")
        if s["initial"] is None:
            final.zero_()
        else:
            final.copy_(s["state"][s["initial"].long()[torch.tensor(order, device="cuda")]])
        y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for t in range(max(n)):
            m = sum(1 for k in n if k > t)
            at = start[:m] + t
            y[at] = token(final[:m], f(s["x"][at]), f(s["dt"][at]), f(s["B"][at]), f(s["C"][at]))
        pool = f(s["state"])
        pool[s["final"].long()[torch.tensor(order, device="cuda")]] = final
        return {"y": y, "state": pool}
    live = s["src"] >= 0
    keep = live.nonzero()[:, 0]
    slot = s["src"][keep].long()
    S = f(_rows(s["state"], slot))
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    T = case["T"]
    if s["op"] == "step":
        for t in range(T):
            y[keep, t] = token(S, f(s["x"][keep, t]), f(s["dt"][keep, t]), f(s["B"][keep, t]), f(s["C"][keep, t]))
        pool = f(s["state"])
        pool[s["dst"][keep].long()] = S
        return {"y": y, "state": pool}
    if s["scale"] is not None:
        S = S * f(s["scale"][slot])[..., None]
    R, start, have = case["R"], s["ring_start"][keep].long(), s["ring_len"][keep].long()
    for i in range(R):  # a row past ring_len changes nothing
        row = (start + i) % R
        use = (i < have).double()
        token(S, f(s["x_cache"][slot, row]), f(s["dt_cache"][slot, row]) * use[:, None], f(s["B_cache"][slot, row]), None)
    caches = {k: f(s[k]) for k in ("x_cache", "B_cache", "dt_cache")}
    for t in range(T):
        y[keep, t] = token(S, f(s["x"][keep, t]), f(s["dt"][keep, t]), f(s["B"][keep, t]), f(s["C"][keep, t]))
        row = (start + have + t) % R
        for k in ("x", "B", "dt"):
            caches[k + "_cache"][slot, row] = f(s[k][keep, t])
    return {"y": y, **caches}
