"""A stack of layers served with the framework's operators: prompts, then rounds of drafted tokens of which a
prefix is accepted, then plain decoding.

A layer is add_rms_norm, a projection to gate, x, B, C and dt, the state space operator, gated_rms_norm and a
projection back.  The operator is ssm_prefill for prompts, replayssm_decode for drafts (the checkpoint state is only
read, the drafts' inputs go to a ring) and ssm_step for tokens that are certain.  A draft that is rejected costs
nothing to undo: its ring rows are written over.  When a ring has no room for another round,
replayssm_materialize moves the accepted rows of all layers into new checkpoints in one call.

    python examples/speculative_decode.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import mamba_replayssm_state_gb300 as rsm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Stack:
    """Layers with random weights and their pools: for each request two state slots, used in turn, and a ring."""

    def __init__(self, layers=4, width=1024, heads=32, groups=2, requests=4, ring=8, state_dtype=F32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.layers, self.width, self.H, self.G, self.dim, self.dstate = layers, width, heads, groups, 64, 128
        self.requests, self.ring, self.inner = requests, ring, heads * 64
        cols = 2 * self.inner + 2 * groups * 128 + heads
        self.w_in = [(rand(width, cols) / width ** 0.5).to(BF16) for _ in range(layers)]
        self.w_out = [(rand(self.inner, width) / self.inner ** 0.5).to(BF16) for _ in range(layers)]
        self.norm = [1.0 + 0.1 * rand(width) for _ in range(layers)]
        self.gate = [1.0 + 0.1 * rand(self.inner) for _ in range(layers)]
        self.bias = [rand(heads) - 3.0 for _ in range(layers)]
        self.A = [-torch.rand(heads, generator=g, device="cuda") - 0.5 for _ in range(layers)]
        self.D = [rand(heads) for _ in range(layers)]
        n, zeros = 2 * requests, lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
        self.state = [zeros(n, heads, 64, 128, dtype=state_dtype) for _ in range(layers)]
        self.rings = [(zeros(n, ring, heads, 64, dtype=BF16), zeros(n, ring, groups, 128, dtype=BF16),
                       zeros(n, ring, heads)) for _ in range(layers)]
        tab, strd = rsm.pointer_table, rsm.stride_table
        self.tables = [tab(self.state), strd(self.state)]
        for i in range(3):
            self.tables += [tab([r[i] for r in self.rings]), strd([r[i] for r in self.rings])]
        self.tables += [tab(self.A), None, None]

    def __call__(self, x, mix):
        """x [rows, width] through the layers; mix(layer, x, dt, B, C) is the state space operator on the rows."""
        residual = torch.zeros(x.shape, dtype=F32, device="cuda")
        for i in range(self.layers):
            x, residual = rsm.add_rms_norm(x, residual, self.norm[i], residual_out=residual)
            z, u, B, C, dt = (x @ self.w_in[i]).split(
                [self.inner, self.inner, self.G * 128, self.G * 128, self.H], dim=-1)
            dt = torch.nn.functional.softplus(dt.float() + self.bias[i])
            y = mix(i, u.unflatten(-1, (self.H, 64)), dt, B.unflatten(-1, (self.G, 128)), C.unflatten(-1, (self.G, 128)))
            y = y.reshape(-1, self.inner)
            x = rsm.gated_rms_norm(y, z, self.gate[i], group_size=self.inner // self.G, out=y) @ self.w_out[i]
        return residual + x.float()

    def prompt(self, x, cu_seqlens, final_slots):
        """Packed prompts x [tokens, width]; their states go to final_slots."""
        return self(x, lambda i, u, dt, B, C: rsm.ssm_prefill(
            u, dt, self.A[i], B, C, cu_seqlens, self.state[i], final_slots=final_slots, D=self.D[i]))

    def draft(self, x, slots, start, have):
        """x [requests, T, width] after the checkpoints and `have` ring rows; the T tokens go to the next rows."""
        b, T = x.shape[:2]
        rows = lambda t: t.unflatten(0, (b, T))  # noqa: E731
        y = self(x.flatten(0, 1), lambda i, u, dt, B, C: rsm.replayssm_decode(
            self.state[i], slots, *self.rings[i], start, have, rows(u), rows(dt), self.A[i], rows(B), rows(C), D=self.D[i]))
        return y.unflatten(0, (b, T))

    def commit(self, slots, new_slots, start, accepted, active):
        """The checkpoints of the active requests, advanced by their accepted ring rows, go to new_slots."""
        every = lambda s: s.expand(self.layers, -1).contiguous()  # noqa: E731
        rsm.replayssm_materialize(
            *self.tables, every(slots), every(new_slots), start, accepted, active, state_dtype=self.state[0].dtype,
            input_dtype=BF16, matrixA_dtype=F32, dim=64, dstate=128, num_heads=self.H, heads_per_group=self.H // self.G,
            max_window=self.ring, ring_buffer_len=self.ring)

    def step(self, x, slots):
        """One certain token a request, x [requests, width]; the states advance in place."""
        return self(x, lambda i, u, dt, B, C: rsm.ssm_step(self.state[i], slots, u, dt, self.A[i], B, C, D=self.D[i]))


def serve(stack, prompts, tokens, drafts=4, accept=None):
    """Prompts (a list of [length, width]), then `tokens` [requests, n, width]: rounds of `drafts` tokens of which
    accept[round][request] are kept (default: all of them) while they last, one by one at the end.  Returns every
    kept token's output, a list of [length + n, width]."""
    b, n = tokens.shape[:2]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [0]
    for p in prompts:
        cu.append(cu[-1] + len(p))
    slots = list(range(b))
    y = stack.prompt(torch.cat(prompts), i32(cu), i32(slots))
    outs = [[y[cu[r]:cu[r + 1]]] for r in range(b)]
    done, start, have = [0] * b, [0] * b, [0] * b  # tokens kept; the ring's first row and rows in use
    turn = 0

    def commit(which):
        if not which:
            return
        new = [(s + b) % (2 * b) for s in slots]
        stack.commit(i32(slots), i32(new), i32(start), i32(have), i32(which + [-1] * (b - len(which))))
        for r in which:  # a ring belongs to its slot: the new one's is empty
            slots[r], start[r], have[r] = new[r], 0, 0

    while min(n - d for d in done) >= drafts:
        commit([r for r in range(b) if have[r] + drafts > stack.ring])
        x = torch.stack([tokens[r, done[r]:done[r] + drafts] for r in range(b)])
        y = stack.draft(x, i32(slots), i32(start), i32(have))
        for r in range(b):
            kept = drafts if accept is None else accept[turn % len(accept)][r]
            outs[r].append(y[r, :kept])
            done[r] += kept
            have[r] += kept
        turn += 1
        if turn > 4 * n:
            raise ValueError("no round accepts a token")
    commit([r for r in range(b) if have[r] > 0])
    while min(done) < n:
        live = [d < n for d in done]
        x = torch.stack([tokens[r, min(done[r], n - 1)] for r in range(b)])
        y = stack.step(x, i32([slots[r] if live[r] else -1 for r in range(b)]))
        for r in range(b):
            if live[r]:
                outs[r].append(y[r:r + 1])
                done[r] += 1
    return [torch.cat(o) for o in outs]


def main():
    torch.manual_seed(1)
    stack = Stack()
    b, n = stack.requests, 21
    prompts = [torch.randn(k, stack.width, device="cuda").to(BF16) for k in (5, 130, 64, 333)]
    tokens = torch.randn(b, n, stack.width, device="cuda").to(BF16)
    outs = serve(stack, prompts, tokens, accept=[[4, 2, 0, 3], [1, 4, 3, 2], [2, 1, 4, 4]])
    whole = [torch.cat([p, t]) for p, t in zip(prompts, tokens)]
    cu = torch.tensor([0] + [len(w) for w in whole], device="cuda").cumsum(0, dtype=torch.int32)
    want = stack.prompt(torch.cat(whole), cu, torch.arange(b, dtype=torch.int32, device="cuda"))
    for r in range(b):
        w = want[cu[r]:cu[r + 1]]
        err = float((outs[r] - w).norm() / w.norm())
        print(f"request {r}: {len(prompts[r])} + {n} tokens, served against one prompt: relative difference {err:.2e}")


if __name__ == "__main__":
    main()
