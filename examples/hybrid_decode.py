"""A hybrid stack served with the framework's operators: state space layers with their short convolution, attention
layers over pages, prompts in pieces, rounds of drafted tokens of which a prefix is accepted, and a request forked.

A state space layer is add_rms_norm, a projection to gate, x | B | C and dt, the short convolution over x | B | C, the
state space operator, gated_rms_norm and a projection back; an attention layer is add_rms_norm, a projection to q, k
and v, rotary_append, paged_attention and a projection back.  What a request has in the convolutions' caches and in the
pages goes by token position, so that rejected drafts are written over; the states are checkpoints with replay rings,
which replayssm_materialize advances by what was accepted.

    python examples/hybrid_decode.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import mamba_replayssm_state_gb300 as rsm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Stack:
    """Layers ("M": state space, "A": attention) with random weights, and their pools for `requests` requests."""

    def __init__(self, layers="MMAMA", width=512, heads=16, groups=2, q_heads=8, kv_heads=2, requests=3, drafts=4, ring=8,
                 page=16, pages=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        proj = lambda a, b: (rand(a, b) / a ** 0.5).to(BF16)  # noqa: E731
        zeros = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.layers, self.width, self.H, self.G, self.QH, self.KH = layers, width, heads, groups, q_heads, kv_heads
        self.inner, self.requests, self.ring, self.page = heads * 64, requests, ring, page
        self.channels = self.inner + 2 * groups * 128
        self.norm = [1.0 + 0.1 * rand(width) for _ in layers]
        self.freq, self.amplitude = rsm.rotary_frequencies(64, 10000.0, scaling="yarn", factor=4.0, original_length=512)
        n = requests
        self.w, self.pools = [], []
        for kind in layers:
            if kind == "M":
                self.w.append(dict(
                    w_in=proj(width, self.inner + self.channels + heads), w_out=proj(self.inner, width),
                    conv=rand(self.channels, 4) / 2, conv_bias=0.1 * rand(self.channels), bias=rand(heads) - 3.0,
                    gate=1.0 + 0.1 * rand(self.inner), A=-torch.rand(heads, generator=g, device="cuda") - 0.5, D=rand(heads)))
                # two state slots a request, used in turn, each with its ring; a convolution's cache keeps what
                # the next tokens look back to, and the drafts
                self.pools.append(dict(
                    conv=zeros(n, 3 + drafts, self.channels), state=zeros(2 * n, heads, 64, 128, t=F32),
                    x=zeros(2 * n, ring, heads, 64), B=zeros(2 * n, ring, groups, 128), dt=zeros(2 * n, ring, heads, t=F32)))
            else:
                self.w.append(dict(w_qkv=proj(width, (q_heads + 2 * kv_heads) * 128), w_out=proj(q_heads * 128, width)))
                self.pools.append(dict(k=zeros(pages, page, kv_heads, 128), v=zeros(pages, page, kv_heads, 128)))
        of = lambda kind, name: [p[name] for k, p in zip(layers, self.pools) if k == kind]  # noqa: E731
        tab = lambda ts: (rsm.pointer_table(ts), rsm.stride_table(ts))  # noqa: E731
        self.tables = [t for name in ("state", "x", "B", "dt") for t in tab(of("M", name))]
        self.tables += [rsm.pointer_table([w["A"] for k, w in zip(layers, self.w) if k == "M"]), None, None]
        self.kv, self.conv = tab(of("A", "k") + of("A", "v")), tab(of("M", "conv"))
        self.table, self.free = torch.full((n, pages), -1, dtype=torch.int32), list(range(pages))
        self.holders = [0] * pages  # requests in whose table a page is
        self.slot = list(range(n))

    def hold(self, r, length):
        """Request r gets the pages that `length` tokens need."""
        for i in range(-(-length // self.page)):
            if self.table[r, i] < 0:
                page = self.free.pop()
                self.table[r, i], self.holders[page] = page, 1

    def release(self, r):
        """Request r gives its pages back: those that no other request holds are free."""
        for page in self.table[r, self.table[r] >= 0].tolist():
            self.holders[page] -= 1
            if self.holders[page] == 0:
                self.free.append(page)
        self.table[r] = -1

    def __call__(self, x, mamba, attend):
        """x [rows, width] through the layers; mamba(i, xBC, dt) and attend(i, q, k, v) work on the rows."""
        residual = torch.zeros(x.shape, dtype=F32, device="cuda")
        for i, kind in enumerate(self.layers):
            w = self.w[i]
            x, residual = rsm.add_rms_norm(x, residual, self.norm[i], residual_out=residual)
            if kind == "M":
                z, xBC, dt = (x @ w["w_in"]).split([self.inner, self.channels, self.H], dim=-1)
                y = mamba(i, xBC, torch.nn.functional.softplus(dt.float() + w["bias"])).reshape(-1, self.inner)
                x = rsm.gated_rms_norm(y, z, w["gate"], group_size=self.inner // self.G) @ w["w_out"]
            else:
                q, k, v = (t.unflatten(-1, (-1, 128)) for t in (x @ w["w_qkv"]).split(
                    [self.QH * 128, self.KH * 128, self.KH * 128], dim=-1))
                x = attend(i, q, k, v).reshape(-1, self.QH * 128) @ w["w_out"]
        return residual + x.float()

    def parts(self, xBC):
        x, B, C = xBC.split([self.inner, self.G * 128, self.G * 128], dim=-1)
        return x.unflatten(-1, (self.H, 64)), B.unflatten(-1, (self.G, 128)), C.unflatten(-1, (self.G, 128))

    def prompt(self, pieces, first):
        """The next tokens of every request, pieces[r] [n, width], after first[r] earlier ones."""
        n = [len(p) for p in pieces]
        cu = [0]
        for r, k in enumerate(n):
            cu.append(cu[-1] + k)
            self.hold(r, first[r] + k)
        cut, slots, lengths = i32(cu), i32(self.slot), i32([f + k for f, k in zip(first, n)])
        table, rows, start = self.table.cuda(), i32(list(range(self.requests))), i32(first)
        fresh = i32([s if f else -1 for s, f in zip(self.slot, first)])

        def mamba(i, xBC, dt):
            w, p = self.w[i], self.pools[i]
            x, B, C = self.parts(rsm.causal_conv(xBC, w["conv"], cut, w["conv_bias"], p["conv"], rows, start))
            return rsm.ssm_prefill(x, dt, w["A"], B, C, cut, p["state"], initial_slots=fresh, final_slots=slots, D=w["D"])

        def attend(i, q, k, v):
            p = self.pools[i]
            q = rsm.rotary_append(q, k, v, self.freq, p["k"], p["v"], table, lengths, cut, amplitude=self.amplitude)
            return torch.cat([rsm.paged_attention(q[None, a:b], p["k"], p["v"], table[r:r + 1], lengths[r:r + 1])[0]
                              for r, (a, b) in enumerate(zip(cu, cu[1:])) if b > a])
        y = self(torch.cat(pieces), mamba, attend)
        return [y[a:b] for a, b in zip(cu, cu[1:])]

    def draft(self, x, first, have):
        """x [requests, T, width] after first[r] tokens, of which have[r] are in the ring."""
        b, T = x.shape[:2]
        for r in range(b):
            self.hold(r, first[r] + T)
        rows = lambda t: t.unflatten(0, (b, T))  # noqa: E731
        request, slots, at, lengths = i32(list(range(b))), i32(self.slot), i32(first), i32([f + T for f in first])
        table, zero, have = self.table.cuda(), i32([0] * b), i32(have)

        def mamba(i, xBC, dt):
            w, p = self.w[i], self.pools[i]
            u, B, C = self.parts(rsm.causal_conv_step(rows(xBC), w["conv"], p["conv"], request, at, w["conv_bias"]))
            return rsm.replayssm_decode(p["state"], slots, p["x"], p["B"], p["dt"], zero, have, u, rows(dt), w["A"], B, C,
                                        D=w["D"])

        def attend(i, q, k, v):
            p = self.pools[i]
            q = rsm.rotary_append(rows(q), rows(k), rows(v), self.freq, p["k"], p["v"], table, lengths,
                                  amplitude=self.amplitude)
            return rsm.paged_attention(q, p["k"], p["v"], table, lengths)
        return self(x.flatten(0, 1), mamba, attend).unflatten(0, (b, T))

    def commit(self, have):
        """Every request's checkpoint advances by its have[r] accepted ring rows, into its other slot."""
        b, count = self.requests, self.layers.count("M")
        new = [(s + b) % (2 * b) for s in self.slot]
        every = lambda s: i32([s] * count)  # noqa: E731
        rsm.replayssm_materialize(
            *self.tables, every(self.slot), every(new), i32([0] * b), i32(have), i32(list(range(b))), state_dtype=F32,
            input_dtype=BF16, matrixA_dtype=F32, dim=64, dstate=128, num_heads=self.H, heads_per_group=self.H // self.G,
            max_window=self.ring, ring_buffer_len=self.ring)
        self.slot = new

    def fork(self, r, to, length):
        """Request `to` becomes a copy of another request r, whose `length` tokens are all committed: full pages are
        shared, the last one, the convolutions' caches and the checkpoints are copied."""
        full = length // self.page
        self.release(to)
        self.table[to, :full] = self.table[r, :full]
        for page in self.table[to, :full].tolist():
            self.holders[page] += 1
        if length % self.page:
            self.hold(to, length)
            p = self.pools[self.layers.index("A")]["k"]
            rsm.copy_pages(*self.kv, i32([int(self.table[r, full])]), i32([int(self.table[to, full])]), dtype=BF16,
                           page_elements=p[0].numel(), num_pages=len(p))
        m = self.pools[self.layers.index("M")]
        rsm.copy_pages(*self.conv, i32([r]), i32([to]), dtype=BF16, page_elements=m["conv"][0].numel(), num_pages=self.requests)
        rsm.copy_pages(self.tables[0], self.tables[1], i32([self.slot[r]]), i32([self.slot[to]]), dtype=F32,
                       page_elements=m["state"][0].numel(), num_pages=2 * self.requests)


def serve(stack, prompts, tokens, cuts, accept, T=4):
    """prompts[r] [n, width] in two pieces, cut at cuts[r]; then tokens [requests, n, width] in rounds of T drafts, of which
    accept[round][r] are kept (what is rejected was another token).  Every kept token's output, [length, width] a
    request; each request has kept the same number."""
    b = stack.requests
    a = stack.prompt([p[:c] for p, c in zip(prompts, cuts)], [0] * b)
    z = stack.prompt([p[c:] for p, c in zip(prompts, cuts)], list(cuts))
    outs, first = [[a[r], z[r]] for r in range(b)], [len(p) for p in prompts]
    done, have = [0] * b, [0] * b
    for kept in accept:
        if max(have) + T > stack.ring:
            stack.commit(have)
            have = [0] * b
        x = torch.stack([tokens[r, done[r]:done[r] + T] for r in range(b)]).clone()
        for r in range(b):
            x[r, kept[r]:] *= -1.0
        y = stack.draft(x, [f + d for f, d in zip(first, done)], have)
        for r in range(b):
            outs[r].append(y[r, :kept[r]])
            done[r] += kept[r]
            have[r] += kept[r]
    stack.commit(have)
    return [torch.cat(o) for o in outs], [f + d for f, d in zip(first, done)]


def main():
    torch.manual_seed(1)
    stack, sizes, accept = Stack(), (37, 150, 64), [[4, 2, 0], [1, 4, 4], [3, 0, 4], [4, 4, 1], [0, 2, 3]]
    rows = lambda n: torch.randn(n, stack.width, device="cuda").to(BF16)  # noqa: E731
    prompts, tokens = [rows(n) for n in sizes], torch.stack([rows(20) for _ in sizes])
    outs, lengths = serve(stack, prompts, tokens, (5, 33, 64), accept)
    whole = [torch.cat([p, t[:n - len(p)]]) for p, t, n in zip(prompts, tokens, lengths)]
    want = Stack().prompt(whole, [0] * 3)
    for r in range(3):
        err = float((outs[r] - want[r]).norm() / want[r].norm())
        print(f"request {r}: {len(whole[r])} tokens, served in pieces against one prompt: relative difference {err:.2e}")
    stack.fork(1, 0, lengths[1])
    a, b = stack.draft(rows(4).expand(3, 4, -1).contiguous(), [lengths[1], lengths[1], lengths[2]], [0] * 3)[:2]
    print(f"request 1 forked: equal outputs {bool(torch.equal(a, b))}")


if __name__ == "__main__":
    main()
