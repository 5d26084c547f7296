"""The operators of hybrid stacks against their definitions in 64 bits.

Bounds.  A rounding is off by at most half a step: U = finfo.eps / 2 of the value (bf16 2^-8, fp32 2^-24).
  convolution  W fused multiply-adds, each within 2^-24 of a sum that is at most m (the sum of the terms' absolute
               values); silu's slope is below 1.1; silu itself within 2^-17 of its value for bf16 (the fast exponential
               and quotient), 2^-20 for fp32 (expf within 2 units, a sum and a quotient, some four 2^-24 in all);
               then the output's rounding.
  rotary       an angle within 2^-24 of a turn, 2 pi 2^-24; sine and cosine within 2^-23, their product with the
               amplitude one rounding more; two products and a sum: 3 2^-24: together below 16 2^-24 of m, the
               amplitude times the pair's absolute values; then the output's rounding.
  attention    a score: dim products and their sums, 2^-23 each of the sum of absolute values (a tensor core may cut
               off where it sums); its product with the scale and the distance from the maximum: two roundings of it,
               2^-22 with room.  A weight's relative error is the score's error
               (and 2^-21 of the exponential), in numerator and denominator: twice that of m, the weights' sum of
               |v|.  The weights' rounding to bf16: U m.  n sums: 2^-23 n m.  Then the output's rounding.
"""
import pytest

torch = pytest.importorskip("torch")

import hybrid_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rand(gen, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def close(got, want, bound):
    got = got.double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0].item()} for {want[bad][0].item()}, bound {bound[bad][0].item()}"


def conv_bound(y, m, W, dtype, silu):
    return U[dtype] * y.abs() * 1.01 + 1.1 * W * E * m + (2.0 ** -17 if dtype == BF16 else 2.0 ** -20) * y.abs() * silu + 1e-30


# ----------------------------------------------------------------------------
# convolution
# ----------------------------------------------------------------------------

LENGTHS = {"one": [1], "few": [37], "block": [32], "edges": [31, 1, 0, 2, 33, 3, 0, 64, 29, 30, 5],
           "ones": [1] * 70, "long": [700, 0, 333]}


def conv_world(C, W, R, n, T, dtype, seed, bias=True, sliced=0):
    g = gen(seed)
    x = rand(g, T, C + sliced, dtype=dtype)
    return (x[:, sliced:], rand(g, C, W, scale=W ** -0.5), rand(g, C, scale=0.3) if bias else None,
            rand(g, n + 1, R, C, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("C,W,R,sliced", [(5376, 4, 4, 0), (1032, 3, 5, 8), (40, 2, 1, 3), (33, 4, 3, 0), (264, 4, 64, 1)])
def test_conv(C, W, R, sliced, lengths, dtype):
    n = LENGTHS[lengths]
    T, cu = sum(n), [0]
    for k in n:
        cu.append(cu[-1] + k)
    x, w, bias, cache = conv_world(C, W, R, len(n), T, dtype, C + T, sliced=sliced)
    slots = [1 + (5 * i) % len(n) if len(n) % 5 else 1 + i for i in range(len(n))]
    pos = [(0, 1, 2, 7, 2 ** 31 - 5)[i % 5] for i in range(len(n))]
    spans = list(zip(cu, cu[1:]))
    y, m, want = ref.conv(x, w, bias, cache, slots, pos, spans, True, W - 1)
    status = word()
    got = rsm.causal_conv(x, w, i32(cu), bias, cache, i32(slots), i32(pos), device_status=status)
    close(got, y, conv_bound(y, m, W, dtype, 1))
    assert torch.equal(cache, want) and int(status) == 0


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_conv_without_a_cache(bias, silu):
    x, w, b, _ = conv_world(100, 4, 4, 0, 90, BF16, 1, bias=bias)
    cu = [0, 50, 50, 90]
    y, m, _ = ref.conv(x, w, b, None, None, None, list(zip(cu, cu[1:])), silu, 0)
    close(rsm.causal_conv(x, w, i32(cu), b, silu=silu), y, conv_bound(y, m, 4, BF16, silu))


def test_conv_pads_and_what_is_out_of_range():
    """A pad, slots past the pool and a negative position: from zero, nothing stored; all but the pad flagged."""
    n = [5, 40, 3, 2, 6]
    cu = [0, 5, 45, 48, 50, 56]
    x, w, b, cache = conv_world(264, 4, 6, 5, 56, BF16, 3)
    before = cache.clone()
    for slots, pos, bit in (([1, -1, 2, 3, 4], [9] * 5, 0), ([1, 6, 2, -7, 4], [9] * 5, 8), ([1, 5, 2, 3, 4], [9, -1, 9, 9, 9], 64)):
        cache.copy_(before)
        live = [s if 0 <= s < 6 and p >= 0 else -1 for s, p in zip(slots, pos)]
        y, m, want = ref.conv(x, w, b, cache, live, pos, list(zip(cu, cu[1:])), True, 3)
        status = word()
        got = rsm.causal_conv(x, w, i32(cu), b, cache, i32(slots), i32(pos), device_status=status)
        close(got, y, conv_bound(y, m, 4, BF16, 1))
        assert torch.equal(cache, want) and int(status) == bit
    assert n[1] > 32


def test_conv_bad_sequences():
    """Sequences outside the tokens, and all from a step back, are skipped: their rows stay."""
    x, w, b, cache = conv_world(264, 4, 6, 9, 60, BF16, 4)
    cu = [-9, -5, 0, 20, 20, 55, 61, 66, 20, 40]
    good = [(0, 0) if not (0 <= a <= e <= 60 and i < 7) else (a, e) for i, (a, e) in enumerate(zip(cu, cu[1:]))]
    slots, pos = list(range(1, 10)), [4] * 9
    y, m, want = ref.conv(x, w, b, cache, slots, pos, good, True, 3)
    out, status = torch.full_like(x, 9.0), word()
    rsm.causal_conv(x, w, i32(cu), b, cache, i32(slots), i32(pos), out=out, device_status=status)
    y[55:] = 9.0
    close(out, y, conv_bound(y, m, 4, BF16, 1))
    assert torch.equal(cache, want) and int(status) == rsm.STATUS_BITS["bad_sequence"]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("batch,T", [(1, 1), (5, 1), (300, 1), (1, 4), (7, 3), (130, 8), (2, 20)])
@pytest.mark.parametrize("C,W,extra,sliced", [(5376, 4, 0, 0), (1032, 3, 2, 8), (40, 2, 0, 3), (33, 4, 9, 0)])
def test_conv_step(C, W, extra, sliced, batch, T, dtype):
    if C == 5376 and batch * T > 400:
        C = 768
    R = W - 1 + T + extra
    x, w, bias, cache = conv_world(C, W, R, batch, batch * T, dtype, C + T + batch, sliced=sliced)
    g = torch.Generator().manual_seed(batch)
    slots = (1 + torch.randperm(batch, generator=g)).tolist()
    if batch > 4:
        slots[2] = -1
    pos = [(0, 1, 2, 11, 2 ** 31 - 1)[i % 5] for i in range(batch)]
    spans = [(i * T, i * T + T) for i in range(batch)]
    y, m, want = ref.conv(x, w, bias, cache, slots, pos, spans, True, T)
    for i, s in enumerate(slots):
        if s < 0:
            y[i * T:i * T + T] = 0
    xx = x.unflatten(0, (batch, T)) if T > 1 else x
    got = rsm.causal_conv_step(xx, w, cache, i32(slots), i32(pos), bias)
    assert got.shape == xx.shape
    close(got.reshape(batch * T, C), y, conv_bound(y, m, W, dtype, 1))
    assert torch.equal(cache, want)


def test_conv_step_out_of_range():
    x, w, b, cache = conv_world(264, 4, 4, 6, 6, BF16, 5)
    before, status = cache.clone(), word()
    got = rsm.causal_conv_step(x, w, cache, i32([1, 7, -1, -2, 3, 4]), i32([3, 3, 3, 3, -2, 3]), b, device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_slot"] | rsm.STATUS_BITS["bad_position"]
    assert bool((got[1:5] == 0).all())
    assert torch.equal(cache[[0, 2, 3, 5, 6]], before[[0, 2, 3, 5, 6]]) and not torch.equal(cache[1], before[1])


def test_conv_in_pieces_with_rejected_drafts():
    """A prompt in two pieces, then drafts of which a part is accepted: the kept tokens' outputs are one prompt's, to
    the bit, since each is the same sums."""
    C, W, T = 264, 4, 5
    x, w, b, cache = conv_world(C, W, W - 1 + T, 2, 60, BF16, 6)
    zero = torch.zeros(2, C, device="cuda", dtype=BF16)
    whole = rsm.causal_conv(x, w, i32([0, 60]), b)
    outs, pos = [], 0
    for n in (2, 31):
        outs.append(rsm.causal_conv(x[pos:pos + n], w, i32([0, n]), b, cache, i32([1]), i32([pos])))
        pos += n
    for k in (3, 0, 5, 1, 4, 2, 5, 5):
        draft = x[pos:pos + T].clone() if pos + T <= 60 else None
        if draft is None:
            break
        draft[k:] = draft[k:] * 2 + 1  # what is rejected was something else
        y = rsm.causal_conv_step(torch.stack([draft, draft]), w, cache, i32([1, 2]), i32([pos, 0]), b)
        outs.append(y[0, :k])
        pos += k
    assert pos > 50
    assert torch.equal(torch.cat(outs), whole[:pos])
    assert bool((zero == 0).all())


# ----------------------------------------------------------------------------
# rotary positions into pages
# ----------------------------------------------------------------------------

def pools(g, pages, page, G, dim, dtype, joined):
    if joined == "rows":  # heads outside rows
        kv = rand(g, pages, 2, G, page, dim, dtype=dtype).transpose(2, 3)
        return kv[:, 0], kv[:, 1]
    if joined:
        kv = rand(g, pages, 2, page, G, dim, dtype=dtype)
        return kv[:, 0], kv[:, 1]
    return rand(g, pages, page, G, dim, dtype=dtype), rand(g, pages, page, G, dim, dtype=dtype)


def rotary_check(q, k, v, freq, spans, lengths, table, kc, vc, interleaved, amplitude, got, before, skipped=()):
    """got (the queries, flat) and the caches against the definition; rows of skipped requests are zero."""
    dtype, page = q.dtype, kc.shape[1]
    wq, wk, wv = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), before[0].double(), before[1].double()
    mq, mk = torch.zeros_like(wq), torch.zeros_like(wk)
    for r, (a, b) in enumerate(spans):
        if a == b or r in skipped:
            continue
        p = torch.arange(lengths[r] - (b - a), lengths[r], device="cuda")
        wq[a:b], mq[a:b] = ref.rotate(q[a:b], p, freq, interleaved, amplitude)
        to = table[r, p // page].long(), p % page
        wk[to], mk[to] = ref.rotate(k[a:b], p, freq, interleaved, amplitude)
        wv[to] = v[a:b].double()
    close(got, wq, U[dtype] * wq.abs() * 1.01 + 16 * E * mq)
    close(kc, wk, torch.where(mk > 0, U[dtype] * wk.abs() * 1.01 + 16 * E * mk, 0.0))
    close(vc, wv, torch.zeros_like(wv))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,G,dim,n", [(8, 2, 128, 64), (6, 3, 64, 16), (4, 4, 128, 12), (5, 1, 72, 36), (2, 1, 10, 3),
                                       (4, 2, 256, 128), (4, 1, 64, 0)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("form", ["one", "window", "packed"])
def test_rotary(form, interleaved, H, G, dim, n, dtype):
    g, h = gen(dim + n), torch.Generator().manual_seed(7)
    page = {"one": 16, "window": 7, "packed": 1 if dim == 64 else 64}[form]
    new = {"one": [1] * 6, "window": [5] * 9, "packed": [0, 1, 129, 3, 0, 40]}[form]
    first = [(0, 3, 4095, 100003, 16, 999999)[i % 6] for i in range(len(new))]
    lengths = [f + m for f, m in zip(first, new)]
    table = torch.full((len(new), max(lengths) // page + 1), -1, dtype=torch.int32)
    free = torch.randperm(sum(m // page + 2 for m in new), generator=h).tolist()
    pages = len(free) + 1
    for r, (a, b) in enumerate(zip(first, lengths)):
        for i in range(a // page, -(-b // page)):
            table[r, i] = free.pop()
    table = table.cuda()
    kc, vc = pools(g, pages, page, G, dim, dtype, {"one": False, "window": True, "packed": "rows"}[form])
    before = kc.clone(), vc.clone()
    T = sum(new)
    q, k, v = rand(g, T, H, dim, dtype=dtype), rand(g, T, G, dim, dtype=dtype), rand(g, T, G, dim, dtype=dtype)
    if dim == 128:
        qkv = torch.cat([t.flatten(1) for t in (q, k, v)], 1)
        q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([H * dim, G * dim, G * dim], 1))
    freq = rand(g, n) if dim == 10 else (10000.0 ** (-torch.arange(n, device="cuda").double() / max(n, 1))).float()
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    lead = (lambda t: t) if form != "window" else (lambda t: t.unflatten(0, (len(new), 5)))
    status = word()
    got = rsm.rotary_append(lead(q), lead(k), lead(v), freq, kc, vc, table, i32(lengths), i32(cu) if form == "packed" else None,
                            interleaved=interleaved, amplitude=1.25, device_status=status)
    assert got.shape == lead(q).shape and got.is_contiguous() and int(status) == 0
    rotary_check(q, k, v, freq, list(zip(cu, cu[1:])), lengths, table, kc, vc, interleaved, 1.25, got.reshape(q.shape), before)


def test_rotary_far_positions():
    """Positions up to the last of 31 bits, on pages of 2^20 tokens: only the last of a request's is looked at."""
    H, G, dim, page = 2, 1, 64, 2 ** 20
    far = [2 ** 31 - 1, 2 ** 24 + 1, 2 ** 30 + 12345]
    q, k, v = rand(gen(1), 3, H, dim), rand(gen(2), 3, G, dim), rand(gen(3), 3, G, dim)
    table = torch.full((3, 2048), -1, dtype=torch.int32)
    for r, p in enumerate(far):
        table[r, (p - 1) // page] = r
    freq, _ = rsm.rotary_frequencies(dim, 10000.0)
    kp, vp = (torch.zeros(3, page, G, dim, device="cuda", dtype=BF16) for _ in range(2))
    qb, kb, vb = q.to(BF16), k.to(BF16), v.to(BF16)
    status = word()
    got = rsm.rotary_append(qb, kb, vb, freq, kp, vp, table.cuda(), i32(far), device_status=status)
    assert int(status) == 0
    for r, p in enumerate(far):
        at = torch.tensor([p - 1], device="cuda")
        wq, mq = ref.rotate(qb[r:r + 1], at, freq, False, 1.0)
        close(got[r:r + 1], wq, U[BF16] * wq.abs() * 1.01 + 16 * E * mq)
        wk, mk = ref.rotate(kb[r:r + 1], at, freq, False, 1.0)
        close(kp[r, (p - 1) % page][None], wk, U[BF16] * wk.abs() * 1.01 + 16 * E * mk)
        assert torch.equal(vp[r, (p - 1) % page], vb[r])
    assert int((vp.flatten(0, 2) != 0).any(1).sum()) == 3


def test_rotary_skipped_and_bad():
    """A request of length 0 (its page entries not looked at), lengths out of range, pages out of range."""
    H, G, dim, page = 4, 2, 64, 8
    q, k, v = rand(gen(1), 6, 2, H, dim, dtype=BF16), rand(gen(2), 6, 2, G, dim, dtype=BF16), rand(gen(3), 6, 2, G, dim, dtype=BF16)
    kc, vc = pools(gen(4), 9, page, G, dim, BF16, False)
    before = kc.clone(), vc.clone()
    freq, _ = rsm.rotary_frequencies(dim)
    lengths = [0, 9, 1, 33, 10, -4]
    table = i32([[99] * 4, [1, 2, -1, -1], [3, 3, 3, 3], [4] * 4, [5, 9, 6, 6], [7] * 4])
    status = word()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_position"] | rsm.STATUS_BITS["bad_page"]
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    # request 4's second page is past the pool: its queries are turned, its keys and values not kept
    spans = [(2 * r, 2 * r + 2) for r in range(6)]
    wq, mq = ref.rotate(q[4], torch.tensor([8, 9], device="cuda"), freq, False, 1.0)
    close(got[4], wq, U[BF16] * wq.abs() * 1.01 + 16 * E * mq)
    rest = got.clone()
    rest[4] = 0
    rotary_check(flat(q), flat(k), flat(v), freq, spans, lengths, table, kc, vc, False, 1.0, flat(rest), before, (0, 2, 3, 4, 5))


def test_rotary_bad_sequences_and_in_place():
    H, G, dim, page = 4, 2, 64, 8
    q, k, v = rand(gen(1), 30, H, dim, dtype=BF16), rand(gen(2), 30, G, dim, dtype=BF16), rand(gen(3), 30, G, dim, dtype=BF16)
    kc, vc = pools(gen(4), 12, page, G, dim, BF16, True)
    before, old = (kc.clone(), vc.clone()), q.clone()
    freq, _ = rsm.rotary_frequencies(dim)
    cu, lengths = [-3, 0, 10, 10, 25, 31, 5, 9], [20] * 7
    table = i32([[r, (r + 1) % 12, (r + 6) % 12] for r in (0, 2, 0, 5, 0, 0, 0)])
    status = word()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32(cu), out=q, device_status=status)
    assert got is q and int(status) == rsm.STATUS_BITS["bad_sequence"]
    spans = [(0, 0), (0, 10), (0, 0), (10, 25), (0, 0), (0, 0), (0, 0)]
    assert torch.equal(q[25:], old[25:])
    want = got.clone()
    want[25:] = 0
    rotary_check(old, k, v, freq, spans, lengths, table, kc, vc, False, 1.0, want, before)


# ----------------------------------------------------------------------------
# attention over pages
# ----------------------------------------------------------------------------

def attention_bound(y, m, top, dim, n, dtype):
    score = top * (dim * 2.0 ** -23 + 2.0 ** -22)
    weight = 2 * (score + 2.0 ** -21) + n * 2.0 ** -23 + (U[BF16] if dtype == BF16 else 0.0)
    return U[dtype] * y.abs() * 1.01 + weight * m


def attention_world(lengths, T, H, G, dim, page, dtype, joined, seed, width=0):
    g = gen(seed)
    table, pages = ref.table(lengths, page, width, torch.Generator().manual_seed(seed))
    kc, vc = pools(g, pages, page, G, dim, dtype, joined)
    return rand(g, len(lengths), T, H, dim, dtype=dtype, scale=2.0), kc, vc, table


def attention_check(q, kc, vc, table, lengths, got, live=None, scale=None):
    live = lengths if live is None else live
    y, m, top = ref.attention(q, kc, vc, table, live, q.shape[-1] ** -0.5 if scale is None else scale)
    close(got, y, attention_bound(y, m, top, q.shape[-1], max(live + [1]), q.dtype))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,G,dim", [(8, 2, 128), (9, 3, 64), (4, 4, 128), (16, 1, 64), (20, 1, 128), (4, 2, 256), (7, 7, 40),
                                     (6, 2, 72), (3, 1, 5), (40, 1, 64)])
@pytest.mark.parametrize("T,page,lengths", [
    (1, 16, [1, 2, 15, 16, 17, 0, 63, 64, 65, 300]), (4, 7, [4, 5, 0, 70, 131]), (2, 1, [2, 33]), (3, 64, [517]),
    (9, 32, [40, 9, 200])])
def test_attention(T, page, lengths, H, G, dim, dtype):
    q, kc, vc, table = attention_world(lengths, T, H, G, dim, page, dtype, page == 7, dim + T + H)
    status = word()
    got = rsm.paged_attention(q, kc, vc, table, i32(lengths), device_status=status)
    attention_check(q, kc, vc, table, lengths, got)
    assert int(status) == 0
    assert bool((got[[i for i, n in enumerate(lengths) if n == 0]] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,G,dim,T,page,lengths,width", [
    (16, 2, 128, 1, 64, [20000], 0), (8, 1, 64, 1, 16, [9000, 1, 4000], 700), (4, 4, 128, 2, 16, [1500] * 20, 0),
    (8, 2, 128, 1, 16, [(37 * i) % 400 for i in range(150)], 0), (4, 2, 256, 1, 32, [3000, 2999], 0),
    (40, 2, 64, 6, 128, [2500, 700], 0)])
def test_attention_long_and_many(H, G, dim, T, page, lengths, width, dtype):
    q, kc, vc, table = attention_world(lengths, T, H, G, dim, page, dtype, False, 5, width)
    attention_check(q, kc, vc, table, lengths, rsm.paged_attention(q, kc, vc, table, i32(lengths)))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256, 40])
def test_attention_strides(dim, dtype):
    """Heads outside rows, queries sliced from a projection (also off 16 bytes), another scale."""
    H, G, T, page, lengths = 6, 2, 3, 16, [100, 3, 65]
    q, kc, vc, table = attention_world(lengths, T, H, G, dim, page, dtype, "rows", dim)
    for off in (0, 1, 8):
        wide = rand(gen(off), 3, T, off + 2 * H * dim, dtype=dtype)
        qs = wide[..., off:off + H * dim].unflatten(-1, (H, dim))
        attention_check(qs, kc, vc, table, lengths, rsm.paged_attention(qs, kc, vc, table, i32(lengths), scale=0.3), scale=0.3)
    # caches off 16 bytes
    n = kc.shape[0] * page * G * dim
    flat = rand(gen(3), 2 * n + 1, dtype=dtype)
    k2, v2 = flat[1:1 + n].view(-1, page, G, dim), flat[1 + n:].view(-1, page, G, dim)
    attention_check(q, k2, v2, table, lengths, rsm.paged_attention(q, k2, v2, table, i32(lengths)))


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 40)])
def test_attention_masked_values(dtype, dim):
    """What a token does not see may be anything: pages nobody holds, rows past the length, later tokens' keys and
    values; and a page out of range is not seen."""
    H, G, T, page, lengths = 8, 2, 4, 16, [70, 5, 200, 4]
    q, kc, vc, table = attention_world(lengths, T, H, G, dim, page, dtype, False, 11)
    kc2, vc2 = torch.full_like(kc, float("nan")), torch.full_like(vc, float("inf"))
    for r, n in enumerate(lengths):
        at = torch.arange(n, device="cuda")
        w = table[r, at // page].long(), at % page
        kc2[w], vc2[w] = kc[w], vc[w]
    attention_check(q, kc, vc, table, lengths, rsm.paged_attention(q, kc2, vc2, table, i32(lengths)))
    # the last token's key and value: no other row may be changed by them
    for bad in (float("nan"), float("inf"), -float("inf")):
        k3, v3 = kc2.clone(), vc2.clone()
        for r, n in enumerate(lengths):
            w = table[r, (n - 1) // page].long(), (n - 1) % page
            k3[w], v3[w] = bad, bad
        want = rsm.paged_attention(q, kc2, vc2, table, i32(lengths))
        got = rsm.paged_attention(q, k3, v3, table, i32(lengths))
        assert torch.equal(got[:, :-1], want[:, :-1])
        assert not bool(got[:, -1].isfinite().any()) or bad < 0
    # pages out of range
    status, t2 = word(), table.clone()
    t2[2, 3], t2[2, 12], t2[1, 0] = kc.shape[0], -1, -5
    got = rsm.paged_attention(q, kc2, vc2, t2, i32(lengths), device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_page"] and bool((got[1] == 0).all())
    attention_check(q, kc, vc, t2, lengths, got)


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 64), (BF16, 24)])
def test_attention_bad_lengths(dtype, dim):
    lengths = [20, -1, 2, 100, 0, 30]
    q, kc, vc, table = attention_world([20, 1, 2, 30, 1, 30], 3, 4, 2, dim, 16, dtype, False, 2, width=3)
    status = word()
    got = rsm.paged_attention(q, kc, vc, table, i32(lengths), device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_position"]
    attention_check(q, kc, vc, table, lengths, got, live=[20, 0, 0, 0, 0, 30])


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 64), (BF16, 24)])
def test_attention_large_scores(dtype, dim):
    """Scores of hundreds, of both signs: the running maximum has to move with them."""
    lengths = [700, 65]
    q, kc, vc, table = attention_world(lengths, 1, 4, 2, dim, 16, dtype, False, 3)
    q = (q.float() * 40).to(dtype)
    attention_check(q, kc, vc, table, lengths, rsm.paged_attention(q, kc, vc, table, i32(lengths)))


# ----------------------------------------------------------------------------
# copies of pages
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,shape,off", [
    (BF16, (16, 2, 128), 0), (F32, (7, 3, 64), 0), (torch.int8, (5, 13), 0), (torch.float16, (1,), 0), (BF16, (100, 333), 0),
    (BF16, (33, 7), 2), (F32, (9, 1031), 1), (torch.float8_e4m3fn, (64, 128), 3)])
def test_copy_pages(dtype, shape, off):
    pages, pools_n, size = 23, 5, 1
    for s in shape:
        size *= s
    es = torch.empty(0, dtype=dtype).element_size()
    g = gen(1)
    raw = torch.randint(0, 255, (pools_n, pages * (size + off) * es + 16), generator=g, device="cuda", dtype=torch.uint8)
    pools_ = [r[:pages * (size + off) * es].view(dtype).as_strided((pages, size), (size + off, 1)) for r in raw]
    src, dst = [3, 20, -1, 7, 3, 9, 23, 5, 5], [0, 1, 2, -1, 4, 9, 6, 30, 8]
    before, status = raw.clone(), word()
    rsm.copy_pages(rsm.pointer_table(pools_), rsm.stride_table(pools_), i32(src), i32(dst), dtype=dtype, page_elements=size,
                   num_pages=pages, device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_page"]
    want = before.clone()
    step = (size + off) * es
    for a, b in ((3, 0), (20, 1), (3, 4), (5, 8)):
        want[:, b * step:b * step + size * es] = before[:, a * step:a * step + size * es]
    assert torch.equal(raw, want)


def test_copy_pages_large():
    """More than a CTA's part of a page, and page offsets past 2^32 bytes."""
    elements, pages = 3 * 2 ** 20 + 40, 1500
    pool = torch.zeros(pages, elements, device="cuda", dtype=torch.int8)
    pool[1400] = torch.randint(-128, 127, (elements,), device="cuda", dtype=torch.int8)
    rsm.copy_pages(rsm.pointer_table([pool]), rsm.stride_table([pool]), i32([1400]), i32([1499]), dtype=torch.int8,
                   page_elements=elements, num_pages=pages)
    assert torch.equal(pool[1499], pool[1400]) and not bool(pool[:1400].any()) and not bool(pool[1401:1499].any())
