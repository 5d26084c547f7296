"""Kernels and branches of the hybrid stacks' operators that a call takes by its size: rotary_append's rings with every
layout, form and kind of bad metadata; attention by single rows past 32-bit offsets, and in place; first calls
from several threads.  Bounds and references are test_hybrid_ops_gpu's."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import hybrid_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402
import test_hybrid_ops_gpu as base  # noqa: E402
from test_hybrid_ops_gpu import BF16, F32, U, E, close, gen, i32, rand, word  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

TYPES = dict(argvalues=[BF16, F32], ids=["bf16", "fp32"])


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ----------------------------------------------------------------------------
# rotary_append's rings: more than 24 tokens an SM of heads turned whole (bf16; 16 of neighbours), more than six of heads turned in part
# ----------------------------------------------------------------------------

def many(dim, turned, interleaved):
    return (24 if turned == dim and not interleaved else 16 if turned == dim else 6) * sms() + 37


def requests(new, page, H, G, dim, dtype, joined, first, seed, slices):
    """Random tokens for requests of new[r] tokens after first[r], and their pages."""
    g, T = gen(seed), sum(new)
    lengths = [f + n for f, n in zip(first, new)]
    table = torch.full((len(new), -(-max(lengths) // page) + 1), -1, dtype=torch.int32)
    free = torch.randperm(sum(n // page + 2 for n in new), generator=torch.Generator().manual_seed(seed)).tolist()
    pages = len(free) + 1
    for r, (a, b) in enumerate(zip(first, lengths)):
        for i in range(a // page, -(-b // page)):
            table[r, i] = free.pop()
    kc, vc = base.pools(g, pages, page, G, dim, dtype, joined)
    q, k, v = (rand(g, T, n, dim, dtype=dtype) for n in (H, G, G))
    if slices:
        q, k, v = (t.unflatten(1, (-1, dim)) for t in torch.cat([t.flatten(1) for t in (q, k, v)], 1).split([H * dim, G * dim, G * dim], 1))
    return q, k, v, kc, vc, table.cuda(), lengths


@pytest.mark.parametrize("dtype", **TYPES)
@pytest.mark.parametrize("joined", [False, True, "rows"])
@pytest.mark.parametrize("form", ["packed", "window"])
@pytest.mark.parametrize("H,G,dim,turned,interleaved", [(6, 3, 64, 64, False), (4, 4, 128, 64, False), (5, 1, 72, 48, True),
                                                        (33, 33, 32, 16, False), (4, 2, 64, 64, True)])
def test_rotary_rings(H, G, dim, turned, interleaved, form, joined, dtype):
    """Keys' and values' heads by one copy or one each (more than a warp's lanes of them), tokens of windows and packed,
    queries to a slice and in place."""
    n = many(dim, turned, interleaved)
    new = [5] * (n // 5 + 1) if form == "window" else [0, 1, n // 2, 3, 0, n - n // 2]
    first = [(0, 3, 4095, 100003, 16, 999999)[i % 6] for i in range(len(new))]
    if form == "window":
        first = [f % 5000 for f in first]
    q, k, v, kc, vc, table, lengths = requests(new, 7 if form == "window" else 64, H, G, dim, dtype, joined, first, dim + H, True)
    freq = rand(gen(3), turned // 2).abs()
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    spans, before, old = list(zip(cu, cu[1:])), (kc.clone(), vc.clone()), q.clone()
    lead = (lambda t: t) if form == "packed" else (lambda t: t.unflatten(0, (len(new), 5)))
    for where in ("new", "slice", "in place"):
        kc.copy_(before[0]), vc.copy_(before[1])
        out = None if where == "new" else q if where == "in place" else torch.zeros(len(q), H + 3, dim, dtype=dtype, device="cuda")[:, 2:H + 2]
        status = word()
        got = rsm.rotary_append(lead(q), lead(k), lead(v), freq, kc, vc, table, i32(lengths), i32(cu) if form == "packed" else None,
                                interleaved=interleaved, amplitude=1.25, out=None if out is None else lead(out), device_status=status)
        assert int(status) == 0
        base.rotary_check(old, k, v, freq, spans, lengths, table, kc, vc, interleaved, 1.25, got.reshape(q.shape), before)


@pytest.mark.parametrize("dtype,dim,turned,interleaved,an_sm", [
    (BF16, 64, 64, False, 24), (BF16, 64, 64, True, 14), (BF16, 64, 32, False, 5), (BF16, 64, 32, True, 5), (BF16, 64, 24, False, 3),
    (BF16, 40, 40, False, 24), (F32, 64, 64, True, 5), (F32, 64, 32, False, 5), (F32, 64, 64, False, 5)])
@pytest.mark.parametrize("more", [0, 1])
def test_rotary_where_rings_begin(dtype, dim, turned, interleaved, an_sm, more):
    """The last number of tokens that have a CTA each, and the first that share rings (but fp32 halves turned whole, which never do)."""
    H, G, n = 3, 1, an_sm * sms() + more
    q, k, v, kc, vc, table, lengths = requests([0, n], 16, H, G, dim, dtype, False, [5, 3], 2, False)
    before, freq = (kc.clone(), vc.clone()), rand(gen(6), turned // 2).abs()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32([0, 0, n]), interleaved=interleaved)
    base.rotary_check(q, k, v, freq, [(0, 0), (0, n)], lengths, table, kc, vc, interleaved, 1.0, got, before)


@pytest.mark.parametrize("dtype", **TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,G,dim,turned,stages", [(128, 16, 256, 128, 2), (96, 8, 256, 128, 3), (64, 8, 256, 64, 5)])
def test_rotary_rings_of_a_whole_sm(H, G, dim, turned, stages, interleaved, dtype):
    """Long tokens, of which two, three and five fit an SM's shared memory (bf16; fp32 heads are half as many)."""
    if dtype == F32:
        H, G = H // 2, G // 2
    place = (H + 2 * G) * dim * (2 if dtype == BF16 else 4) + 4 * turned
    assert 3 * place > 104 * 1024 and 216 * 1024 // place == stages
    n = 6 * sms() + 40
    new = [n // 3, 0, n - n // 3]
    q, k, v, kc, vc, table, lengths = requests(new, 64, H, G, dim, dtype, False, [9, 0, 70000], 5, False)
    freq, before = rand(gen(4), turned // 2).abs(), (kc.clone(), vc.clone())
    lengths[0] = 0  # skipped: its rows are zero
    cu = [0, new[0], new[0], n]
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32(cu), interleaved=interleaved)
    base.rotary_check(q, k, v, freq, list(zip(cu, cu[1:])), lengths, table, kc, vc, interleaved, 1.0, got, before, (0,))


@pytest.mark.parametrize("dtype", **TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_rings_skipped_and_bad(interleaved, dtype):
    """Requests of length 0 (their pages not looked at), lengths and pages out of range, among many that are good."""
    H, G, dim, page, T = 4, 2, 64, 8, 2
    b = many(dim, 32, interleaved) // T + 1
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(2, 33, (b,), generator=g).tolist()
    table = torch.arange(4 * b, dtype=torch.int32).view(b, 4)
    kc, vc = base.pools(gen(4), 4 * b, page, G, dim, dtype, "rows")
    skipped, lost = [], []
    for r in range(0, b, 3):
        kind = r // 3 % 5
        if kind == 4:
            lost.append(r)
            lengths[r] = 8 * (1 + r % 4)
            table[r, r % 4] = (-1, 4 * b, 2 ** 31 - 1)[r // 15 % 3]  # the page of both new tokens
        else:
            skipped.append(r)
            lengths[r] = (0, 33, -4, 1)[kind]
            if kind == 0:
                table[r] = 2 ** 30
    table = table.cuda()
    q, k, v = (rand(gen(i), b, T, n, dim, dtype=dtype) for i, n in ((1, H), (2, G), (3, G)))
    freq, before, status = rand(gen(5), 16).abs(), (kc.clone(), vc.clone()), word()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), interleaved=interleaved, device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_position"] | rsm.STATUS_BITS["bad_page"]
    flat, rest = (lambda t: t.flatten(0, 1)), got.clone()
    for r in lost:  # turned, and not kept
        wq, mq = ref.rotate(q[r], torch.arange(lengths[r] - T, lengths[r], device="cuda"), freq, interleaved, 1.0)
        close(got[r], wq, U[dtype] * wq.abs() * 1.01 + 16 * E * mq)
    rest[lost] = 0
    assert bool((got[skipped] == 0).all())
    base.rotary_check(flat(q), flat(k), flat(v), freq, [(T * r, T * r + T) for r in range(b)], lengths, table, kc, vc,
                      interleaved, 1.0, flat(rest), before, skipped + lost)


@pytest.mark.parametrize("dtype", **TYPES)
def test_rotary_rings_bad_sequences_in_place(dtype):
    """Sequences outside the tokens and all from a step back: their rows stay."""
    H, G, dim, page = 4, 2, 64, 8
    n = many(dim, 32, False)
    cu = [-3, 0, n // 2, n // 2, n - 9, n + 1, 5, 9]
    spans = [(0, 0), (0, n // 2), (0, 0), (n // 2, n - 9), (0, 0), (0, 0), (0, 0)]
    new = [b - a for a, b in spans]
    q, k, v, kc, vc, table, lengths = requests(new, page, H, G, dim, dtype, True, [0, 11, 0, 2000, 0, 0, 0], 7, False)
    tokens = [torch.cat([t, rand(gen(i), 9, t.shape[1], dim, dtype=dtype)]) for i, t in enumerate((q, k, v))]
    q, k, v = tokens
    assert len(q) == n
    before, old, freq = (kc.clone(), vc.clone()), q.clone(), rand(gen(5), 16).abs()
    status = word()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32(cu), out=q, device_status=status)
    assert got is q and int(status) == rsm.STATUS_BITS["bad_sequence"]
    assert torch.equal(q[n - 9:], old[n - 9:])
    want = got.clone()
    want[n - 9:] = 0
    base.rotary_check(old, k, v, freq, spans, lengths, table, kc, vc, False, 1.0, want, before)


def test_rotary_rings_captured_and_replayed():
    """A captured call of many tokens reads lengths and tokens when it is replayed."""
    H, G, dim, page, T = 4, 2, 64, 16, 4
    b = many(dim, 32, False) // T + 1
    kc, vc = base.pools(gen(4), 4 * b, page, G, dim, BF16, False)
    before = kc.clone(), vc.clone()
    table = torch.arange(4 * b, device="cuda", dtype=torch.int32).view(b, 4)
    q, k, v = (rand(gen(i), b, T, n, dim, dtype=BF16) for i, n in ((1, H), (2, G), (3, G)))
    lengths, freq = i32([4 + i % 61 for i in range(b)]), rand(gen(5), 16).abs()
    rsm.rotary_append(q, k, v, freq, kc, vc, table, lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rsm.rotary_append(q, k, v, freq, kc, vc, table, lengths)
    lengths.copy_(i32([64 - i % 50 if i % 7 else 0 for i in range(b)]))
    q.copy_(rand(gen(8), b, T, H, dim, dtype=BF16))
    kc.copy_(before[0]), vc.copy_(before[1])
    graph.replay()
    n, flat = lengths.tolist(), (lambda t: t.flatten(0, 1))
    base.rotary_check(flat(q), flat(k), flat(v), freq, [(T * r, T * r + T) for r in range(b)], n, table, kc, vc, False, 1.0,
                      flat(got), before, [r for r in range(b) if n[r] == 0])


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------

def test_attention_by_single_rows_past_2_31_values():
    """Pages whose offsets pass 32 bits where neither boxes (pages of 8) nor gathers (padded heads) load them."""
    G, dim, n, page = 16, 72, 300, 8
    pages = 2 ** 31 // (page * G * dim) + 40
    kc, vc = (torch.zeros(pages, page, G, dim, device="cuda", dtype=BF16) for _ in range(2))
    need = -(-n // page)
    at = torch.arange(pages - need, pages, device="cuda")
    kc[at], vc[at] = rand(gen(1), need, page, G, dim, dtype=BF16), rand(gen(2), need, page, G, dim, dtype=BF16)
    q = rand(gen(3), 1, 1, 32, dim, dtype=BF16, scale=2.0)
    got = rsm.paged_attention(q, kc, vc, at[None].int(), i32([n]))
    few = torch.arange(need, device="cuda", dtype=torch.int32)[None]
    k2, v2 = kc[at].clone(), vc[at].clone()
    assert torch.equal(got, rsm.paged_attention(q, k2, v2, few, i32([n])))
    base.attention_check(q, k2, v2, few, [n], got)


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128), (BF16, 20), (BF16, 72)])
@pytest.mark.parametrize("T", [1, 4, 9, 40])
def test_attention_in_place(T, dtype, dim):
    """out may be q: long requests, which several CTAs share, and short ones, skipped ones among them."""
    lengths = [3000, T, 0, 130, 64 + T, 1000]
    q, kc, vc, table = base.attention_world(lengths, T, 8, 2, dim, 16, dtype, False, dim + T)
    want, mine = rsm.paged_attention(q, kc, vc, table, i32(lengths)), q.clone()
    assert rsm.paged_attention(mine, kc, vc, table, i32(lengths), out=mine) is mine
    assert torch.equal(mine, want)


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128), (F32, 256)])
@pytest.mark.parametrize("odd", [40.0, float("inf"), float("nan")])
def test_attention_rows_do_not_depend_on_one_another(odd, dtype, dim):
    """A head whose scores are large, or no numbers, leaves the bits of the others as they are."""
    lengths = [700, 65, 3, 200] * 20
    q, kc, vc, table = base.attention_world(lengths, 2, 8, 2, dim, 16, dtype, False, dim)
    want = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    q[:, :, 5] *= odd
    got = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    others = [h for h in range(8) if h != 5]
    assert torch.equal(got[:, :, others], want[:, :, others])


# ----------------------------------------------------------------------------
# first calls
# ----------------------------------------------------------------------------

FIRST = """
import sys, threading
import torch
sys.path[:0] = sys.argv[1:3]
import mamba_replayssm_state_gb300 as rsm
import test_hybrid_paths_gpu as paths

def calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, t=torch.bfloat16: torch.randn(s, generator=g, device="cuda").to(t)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, lengths = torch.arange(30, device="cuda", dtype=torch.int32).view(3, 10), i(100, 3, 70)
    out = []
    for t in (torch.bfloat16, torch.float32):
        for dim in (64, 128, 256):
            for T in (1, 3, 7):
                q, k, v = r(3, T, 8, dim, t=t), r(30, 16, 2, dim, t=t), r(30, 16, 2, dim, t=t)
                out.append(lambda q=q, k=k, v=v: rsm.paged_attention(q, k, v, table, lengths))
        n = 6 * paths.sms() + 9
        q, k, v, kc, vc = r(n, 4, 64, t=t), r(n, 2, 64, t=t), r(n, 2, 64, t=t), r(n, 1, 2, 64, t=t), r(n, 1, 2, 64, t=t)
        f, at, cu, total = r(16, t=torch.float32), torch.arange(n, device="cuda", dtype=torch.int32)[None], i(0, n), i(n)
        out.append(lambda q=q, k=k, v=v, kc=kc, vc=vc, f=f, at=at, cu=cu, total=total:
                   rsm.rotary_append(q, k, v, f, kc.clone(), vc.clone(), at, total, cu))
        x, w, c = r(40, 264, t=t), r(264, 4, t=torch.float32), r(4, 6, 264, t=t)
        out.append(lambda x=x, w=w, c=c: rsm.causal_conv(x, w, i(0, 1, 33, 40), None, c.clone(), i(2, 0, 1), i(0, 2, 7)))
        out.append(lambda x=x, w=w, c=c: rsm.causal_conv_step(x[:3], w, c.clone(), i(2, 0, 1), i(0, 2, 7)))
    torch.cuda.synchronize()
    return out

todo, together, got, failed = calls(), threading.Barrier(4), [None] * 4, []

def work(n):
    try:
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            together.wait()
            got[n] = [f() for f in todo]
            torch.cuda.current_stream().synchronize()
    except BaseException as e:
        failed.append(repr(e))
        together.abort()

threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
want = [f() for f in todo]
for mine in got:
    assert all(torch.equal(a, b) for a, b in zip(mine, want))
print("the same", len(want))
"""


def test_first_calls_from_several_threads():
    """Every kernel's first call comes from four threads at once, in a process of its own."""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST, os.path.dirname(here), here], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "the same 24" in r.stdout, r.stdout + r.stderr
