"""The operators of hybrid stacks where a call's sizes, values or callers are unusual.  Bounds and references are
test_hybrid_ops_gpu's, or stated at the test."""
import threading

import pytest

torch = pytest.importorskip("torch")

import hybrid_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402
import test_hybrid_ops_gpu as base  # noqa: E402
from mamba_replayssm_state_gb300 import hybrid  # noqa: E402
from test_hybrid_ops_gpu import BF16, F32, close, gen, i32, rand, word  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def calls(dtype=BF16, dim=64, seed=1):
    """Every operator on small tensors: (function of the keyword arguments, its tensors by name, those it writes)."""
    g = gen(seed)
    C, b, T, H, G, page = 264, 3, 2, 4, 2, 16
    conv = dict(x=rand(g, 40, C, dtype=dtype), weight=rand(g, C, 4), cu_seqlens=i32([0, 1, 33, 40]), bias=rand(g, C),
                cache=rand(g, b, 6, C, dtype=dtype), slots=i32([2, 0, 1]), positions=i32([0, 2, 7]))
    step = dict(x=rand(g, b, T, C, dtype=dtype), weight=rand(g, C, 4), cache=rand(g, b, 6, C, dtype=dtype),
                slots=i32([1, 2, 0]), positions=i32([0, 5, 9]), bias=rand(g, C))
    lengths, table = i32([100, 3, 70]), ref.table([100, 3, 70], page, 8, torch.Generator().manual_seed(1))
    pages = dict(k_cache=rand(g, table[1], page, G, dim, dtype=dtype), v_cache=rand(g, table[1], page, G, dim, dtype=dtype),
                 page_table=table[0], lengths=lengths)
    rot = dict(q=rand(g, b, T, H, dim, dtype=dtype), k=rand(g, b, T, G, dim, dtype=dtype), v=rand(g, b, T, G, dim, dtype=dtype),
               inv_freq=rand(g, dim // 2).abs(), **{k: v.clone() for k, v in pages.items()})
    att = dict(q=rand(g, b, T, H, dim, dtype=dtype), **pages)
    return {"causal_conv": (rsm.causal_conv, conv, ["cache"]), "causal_conv_step": (rsm.causal_conv_step, step, ["cache"]),
            "rotary_append": (rsm.rotary_append, rot, ["k_cache", "v_cache"]), "paged_attention": (rsm.paged_attention, att, [])}


NAMES = ["causal_conv", "causal_conv_step", "rotary_append", "paged_attention"]


def run(name, change=None, **kw):
    """(output, tensors written) of the operator on fresh tensors; `change`: {argument: tensor}."""
    f, t, written = calls()[name]
    t = t | (change or {})
    return f(**t, **kw), [t[n] for n in written]


def same(a, b):
    return torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[1], b[1]))


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_into_the_library(name):
    """The C++ side's calls and Python's give the same bits: results allocated or passed, a status word, a stream."""
    want = run(name)
    assert same(run(name, out=torch.empty_like(want[0])), want)
    status = word()
    assert same(run(name, device_status=status), want) and int(status) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = run(name, stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


def off(t):
    """t an element further on than an allocation starts."""
    moved = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    return moved.copy_(t)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("name", NAMES)
def test_tensors_at_any_address(name, dtype):
    """Each tensor, results among them, may start at any element.

    Other paths may serve such a call, and two results of one formula differ by two roundings, a step:
    2 (eps / 2) |y|.  Beside them, for values around 1: sums of few fp32 terms, 1e-5; attention in fp32, whose
    scores are off by 64 2^-24 sum |q k| / 8 (3e-5 where that sum is 60), on two sides, in the numerator and the
    denominator, times |v| up to 4: 5e-4; and with bf16 weights 2^-8 of the largest |v|."""
    f, t, written = calls(dtype)[name]
    first = {k: v.clone() for k, v in t.items()}
    want, kept = f(**first), [first[n] for n in written]
    atol = 1e-5 if name != "paged_attention" else 5e-4 if dtype == F32 else 2.0 ** -8 * float(t["v_cache"].abs().max())
    tol = dict(rtol=torch.finfo(dtype).eps, atol=atol)
    for which in (*t, "out"):
        args = {k: off(v) if k == which else v.clone() for k, v in t.items()}
        if which == "out":
            room = torch.full((want.numel() + 17,), 7.0, dtype=dtype, device="cuda")
            for at in (1, 2, 4):
                room.fill_(7.0)
                args = {k: v.clone() for k, v in t.items()}
                out = room[at:at + want.numel()].view(want.shape)
                assert f(**args, out=out) is out
                torch.testing.assert_close(out, want, **tol)
                assert bool((room[:at] == 7.0).all()) and bool((room[at + want.numel():] == 7.0).all())
        else:
            torch.testing.assert_close(f(**args), want, **tol)
        for n, k in zip(written, kept):
            torch.testing.assert_close(args[n], k, **tol)


@pytest.mark.parametrize("dtype,dim,T", [(BF16, 128, 4), (BF16, 256, 1), (F32, 128, 1), (F32, 64, 9), (BF16, 24, 1)])
def test_attention_outputs_at_any_address(dtype, dim, T):
    """The stores of units in one piece and of those in several, heads of every compiled size."""
    lengths = [9000, 40, 70, 0, 64]
    q, kc, vc, table = base.attention_world(lengths, T, 8, 2, dim, 16, dtype, True, 31)
    want = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    for at in (1, 2, 4, 8):
        room = torch.full((want.numel() + 17,), 7.0, dtype=dtype, device="cuda")
        out = room[at:at + want.numel()].view(want.shape)
        assert torch.equal(rsm.paged_attention(q, kc, vc, table, i32(lengths), out=out), want)
        assert bool((room[:at] == 7.0).all()) and bool((room[at + want.numel():] == 7.0).all())


@pytest.mark.parametrize("name", NAMES)
def test_a_raw_stream_needs_results(name):
    side = torch.cuda.Stream()
    with pytest.raises(ValueError, match="raw stream"):
        run(name, stream=side.cuda_stream)


@pytest.mark.parametrize("name", ["causal_conv", "causal_conv_step"])
@pytest.mark.parametrize("pad", [2 ** 32 - 1, 2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_a_pad_slot_past_32_bits_is_refused(name, pad):
    with pytest.raises(ValueError, match="pad_slot_id"):
        run(name, pad_slot_id=pad)


@pytest.mark.parametrize("name,args", [("causal_conv", ["x", "weight", "bias", "cache"]),
                                       ("causal_conv_step", ["x", "weight", "bias", "cache"]),
                                       ("rotary_append", ["q", "k", "v", "inv_freq", "k_cache", "v_cache"]),
                                       ("paged_attention", ["q", "k_cache", "v_cache"])])
def test_a_gradient_that_would_be_lost_is_refused(name, args):
    want = run(name)
    for arg in args:
        t = {arg: calls()[name][1][arg].clone().requires_grad_()}
        for way in ({}, {"out": torch.empty_like(want[0])}):
            with pytest.raises(ValueError, match="forward only"):
                run(name, t, **way)
            with torch.no_grad():
                t[arg] = calls()[name][1][arg].clone().requires_grad_()
                assert same(run(name, t, **way), want)


@pytest.mark.parametrize("name,change,msg", [
    ("causal_conv", dict(cache=lambda t: t["cache"][:1].expand(3, 6, 264)), "overlap"),
    ("causal_conv_step", dict(cache=lambda t: t["cache"][:1].expand(3, 6, 264)), "overlap"),
    ("causal_conv", dict(cache=lambda t: t["cache"].float()), "cache must be"),
    ("causal_conv", dict(slots=lambda t: None, positions=lambda t: None), "go together"),
    ("causal_conv", dict(cache=lambda t: None, slots=lambda t: None), "positions need a cache"),
    ("causal_conv", dict(cache=lambda t: t["cache"][:, :2].contiguous()), "cache_rows"),
    ("causal_conv_step", dict(cache=lambda t: t["cache"][:, :4].contiguous()), "cache_rows"),
    ("causal_conv", dict(weight=lambda t: t["weight"].repeat(1, 2)), "width"),
    ("causal_conv_step", dict(slots=lambda t: t["slots"].long()), "slots must be"),
    ("causal_conv_step", dict(positions=lambda t: t["positions"][:2]), "positions must be"),
    ("rotary_append", dict(k_cache=lambda t: t["k_cache"][:1].expand_as(t["k_cache"])), "overlap"),
    ("rotary_append", dict(k_cache=lambda t: t["k_cache"].as_strided(t["k_cache"].shape, (64, 128, 64, 1))), "overlap"),
    ("paged_attention", dict(v_cache=lambda t: t["v_cache"].as_strided(t["v_cache"].shape, (2048, 64, 64, 1))), "overlap"),
    ("rotary_append", dict(v_cache=lambda t: t["v_cache"][:, :8]), "one shape"),
    ("rotary_append", dict(inv_freq=lambda t: torch.ones(33, device="cuda")), "rotary_dim"),
    ("paged_attention", dict(k_cache=lambda t: t["k_cache"].transpose(2, 3).contiguous().transpose(2, 3)), "contiguous"),
    ("paged_attention", dict(page_table=lambda t: t["page_table"].long()), "page_table must be"),
    ("paged_attention", dict(page_table=lambda t: t["page_table"].t().contiguous().t()), "page_table must be"),
    ("paged_attention", dict(page_table=lambda t: t["page_table"][:2]), "page_table must be"),
    ("paged_attention", dict(lengths=lambda t: t["lengths"].long()), "lengths must be"),
    ("paged_attention", dict(q=lambda t: t["q"][:, :, :3].contiguous()), "num_kv_heads"),
    ("paged_attention", dict(k_cache=lambda t: t["k_cache"].float()), "k_cache must be")])
def test_refusals(name, change, msg):
    t = calls()[name][1]
    with pytest.raises((ValueError, rsm.ReplaySSMError), match=msg):
        run(name, {k: f(t) for k, f in change.items()})


@pytest.mark.parametrize("n", [2 ** 63, -2 ** 70])
def test_a_page_past_64_bits_is_refused(n):
    t = torch.zeros(2, 8, device="cuda")
    with pytest.raises(ValueError, match="64 bits"):
        rsm.copy_pages(rsm.pointer_table([t]), rsm.stride_table([t]), i32([0]), i32([1]), dtype=F32, page_elements=n, num_pages=2)


def test_results_that_overlap_are_refused():
    t = calls()["causal_conv"][1]
    with pytest.raises(rsm.ReplaySSMError, match="out must not be x"):
        rsm.causal_conv(**t, out=t["x"])
    with pytest.raises(ValueError, match="rows of out overlap"):
        rsm.causal_conv(**t, out=torch.empty(264, device="cuda", dtype=BF16).expand(40, 264))
    t = calls()["rotary_append"][1]
    with pytest.raises(ValueError, match="overlap"):
        rsm.rotary_append(**t, out=torch.empty(4, 64, device="cuda", dtype=BF16).expand(3, 2, 4, 64))


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed_on_changed_inputs(name):
    """A captured call reads its tensors when it is replayed: other values, and other lengths and positions."""
    f, t, written = calls()[name]
    keep = {k: v.clone() for k, v in t.items()}
    f(**t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f(**t)
    other = calls(seed=5)[name][1]
    for change in ({}, dict(positions=i32([3, 0, 1])), dict(lengths=i32([2, 90, 0])), dict(lengths=i32([128, 128, 128]))):
        for k in t:
            if k not in ("page_table", "cu_seqlens", "slots"):
                t[k].copy_(change.get(k, other[k] if change else keep[k]))
        if "page_table" in t:
            t["page_table"].copy_(torch.arange(24, device="cuda", dtype=torch.int32).view(3, 8) % t["k_cache"].shape[0])
            if name == "rotary_append":  # (requests write to pages of their own)
                t["page_table"].copy_(torch.arange(3, device="cuda", dtype=torch.int32)[:, None].expand(3, 8))
        fresh = {k: v.clone() for k, v in t.items()}
        graph.replay()
        want = f(**fresh)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(t[n], fresh[n]) for n in written), change


def test_calls_from_two_threads_on_their_streams():
    """Each thread's calls get what they get alone, whichever kernel is set up first."""
    want = {n: run(n) for n in NAMES}
    wrong = []

    def work():
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            for k in range(60):
                for n in NAMES:
                    got = run(n)
                    torch.cuda.current_stream().synchronize()
                    if not same(got, want[n]):
                        wrong.append((n, k))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


# ----------------------------------------------------------------------------
# convolution
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("C", [264, 33])
def test_conv_values_of_other_sequences_do_not_matter(C):
    """NaN in a neighbour's tokens, in rows outside every sequence, in cache rows of no use and in other slots."""
    nan = float("nan")
    cu = [0, 9, 50, 50, 51, 90]
    x, w, b, cache = base.conv_world(C, 4, 6, 5, 100, BF16, 3)
    pos = [0, 2, 5, 1, 3]
    x[9:50] = nan
    x[90:] = nan
    cache[2:] = nan
    cache[1, [r for r in range(6) if r not in (9 % 6, 8 % 6, 7 % 6)]] = nan  # (position 0: nothing is looked up)
    cache[4, 0] = 1.0  # position 1 looks back to row 0 only
    cache[5, [0, 1, 2]] = 0.5
    y, m, want = ref.conv(x, w, b, cache, [1, 2, 3, 4, 5], pos, list(zip(cu, cu[1:])), True, 3)
    out = torch.full_like(x, 7.0)
    rsm.causal_conv(x, w, i32(cu), b, cache, i32([1, 2, 3, 4, 5]), i32(pos), out=out)
    good = [i for i in range(90) if not 9 <= i < 50]
    close(out[good], y[good], base.conv_bound(y, m, 4, BF16, 1)[good])
    assert bool((out[90:] == 7).all()) and bool(out[9:50].isnan().all())
    assert torch.equal(cache.isnan(), want.isnan()) and torch.equal(cache.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("C", [264, 33])
@pytest.mark.parametrize("cu", [[70, 75, 90], [1, 1, 3], [95, 96, 100], [47, 50, 51], [3, 3, 3], [0, 0, 100]])
def test_conv_rows_outside_the_sequences(C, cu):
    """Tokens before the first sequence and behind the last are nobody's: their rows stay, and a sequence is read and
    its inputs are stored once, wherever blocks of tokens begin."""
    x, w, b, cache = base.conv_world(C, 4, 3, 2, 100, BF16, 3)
    spans = list(zip(cu, cu[1:]))
    y, m, want = ref.conv(x, w, b, cache, [1, 2], [4, 7], spans, True, 3)
    out, status = torch.full_like(x, 7.0), word()
    rsm.causal_conv(x, w, i32(cu), b, cache, i32([1, 2]), i32([4, 7]), out=out, device_status=status)
    inside = [i for a, e in spans for i in range(a, e)]
    close(out[inside], y[inside], base.conv_bound(y, m, 4, BF16, 1)[inside])
    outside = [i for i in range(100) if i not in inside]
    assert bool((out[outside] == 7).all()) and torch.equal(cache, want) and int(status) == 0


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_conv_extreme_values(dtype):
    """silu far out: large inputs come through, large negative ones are -0 or tiny; infinities as the formula has it."""
    big = 3e38 if dtype == F32 else 3e38
    x = torch.tensor([[0.0], [100.0], [-100.0], [1e4], [-1e4], [big], [-big], [float("inf")]], device="cuda").to(dtype).repeat(1, 8)
    w = torch.zeros(8, 4, device="cuda")
    w[:, 3] = 1.0
    y = rsm.causal_conv(x, w, i32([0, 8]))
    v = x.double()
    want = v * torch.sigmoid(v)
    ok = want.isfinite()
    close(torch.where(ok, y, 0), torch.where(ok, want, 0.0), 2.0 ** -7 * want.abs().nan_to_num(0, 0, 0) * (1 if dtype == BF16 else 2.0 ** -12) + 1e-30)
    assert bool((y[7] == float("inf")).all() | y[7].isnan().all())


def test_conv_positions_wrap_in_the_cache():
    """A step at every phase of a ring of seven rows equals one prompt."""
    x, w, b, cache = base.conv_world(264, 4, 7, 1, 40, BF16, 9)
    whole = rsm.causal_conv(x, w, i32([0, 40]), b)
    outs = [rsm.causal_conv_step(x[t:t + 1], w, cache, i32([1]), i32([t]), b) for t in range(40)]
    assert torch.equal(torch.cat(outs), whole)


def test_conv_more_than_2_31_values():
    """A cache and a prompt whose offsets pass 32 bits; only the ends are looked at."""
    C, R = 32768, 8
    S = 2 ** 31 // (C * R) + 3
    cache = torch.zeros(S, R, C, device="cuda", dtype=BF16)
    T = 2 ** 31 // C + 37
    x = torch.zeros(T, C, device="cuda", dtype=BF16)
    x[-20:] = rand(gen(1), 20, C, dtype=BF16)
    cache[S - 1] = rand(gen(2), R, C, dtype=BF16)
    before = cache[S - 1].clone()
    w, b = rand(gen(3), C, 4), rand(gen(4), C)
    y = rsm.causal_conv(x, w, i32([0, T - 20, T]), b, cache, i32([-1, S - 1]), i32([0, 5]))
    small = before[None].clone()
    want = rsm.causal_conv(x[-20:].clone(), w, i32([0, 20]), b, small, i32([0]), i32([5]))
    assert torch.equal(y[-20:], want) and torch.equal(cache[S - 1], small[0])
    got = rsm.causal_conv_step(x[-1:], w, cache, i32([S - 1]), i32([25]), b)
    assert torch.equal(got, rsm.causal_conv_step(x[-1:].clone(), w, small, i32([0]), i32([25]), b))


# ----------------------------------------------------------------------------
# rotary
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [1, 2431, 2433, 5000])
def test_rotary_few_and_many_tokens(tokens):
    """The two kernels, skipped requests among them."""
    H, G, dim, n, page = 4, 2, 64, 32, 64
    b = 3 if tokens > 3 else 1
    cu = [0, tokens // 3, tokens // 3, tokens] if b == 3 else [0, 1]
    new = [q - p for p, q in zip(cu, cu[1:])]
    lengths = [7 + m for m in new]
    table, pages = ref.table(lengths, page, 0, torch.Generator().manual_seed(1))
    if b == 3:
        lengths[0] = 0
    g = gen(tokens)
    kc, vc = base.pools(g, pages, page, G, dim, BF16, True)
    before = kc.clone(), vc.clone()
    q, k, v = rand(g, tokens, H, dim, dtype=BF16), rand(g, tokens, G, dim, dtype=BF16), rand(g, tokens, G, dim, dtype=BF16)
    freq, _ = rsm.rotary_frequencies(2 * n)
    status = word()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32(cu), device_status=status)
    assert int(status) == 0
    base.rotary_check(q, k, v, freq, list(zip(cu, cu[1:])), lengths, table, kc, vc, False, 1.0, got, before,
                      (0,) if b == 3 else ())


@pytest.mark.parametrize("turned,an_sm", [(64, 24), (32, 6)])
@pytest.mark.parametrize("more", [0, 1])
def test_rotary_where_the_kernels_take_turns(turned, an_sm, more):
    """The last number of tokens that have a CTA each, and the first that share rings, of one request and empty ones."""
    tokens = an_sm * torch.cuda.get_device_properties(0).multi_processor_count + more
    H, G, dim, page = 3, 1, 64, 16
    cu, lengths = [0, 0, tokens, tokens], [5, tokens + 3, 1]
    table, pages = ref.table(lengths, page, 0, torch.Generator().manual_seed(1))
    g = gen(tokens)
    kc, vc = base.pools(g, pages, page, G, dim, BF16, False)
    before = kc.clone(), vc.clone()
    q, k, v = (rand(g, tokens, n, dim, dtype=BF16) for n in (H, G, G))
    freq = rand(g, turned // 2).abs()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32(cu))
    base.rotary_check(q, k, v, freq, list(zip(cu, cu[1:])), lengths, table, kc, vc, False, 1.0, got, before)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,turned", [(128, 24), (64, 8), (64, 16), (128, 20), (40, 40), (128, 6), (96, 0), (36, 24), (256, 120)])
def test_rotary_widths_of_the_pairs(dim, turned, interleaved, dtype):
    """Halves of whole 16 bytes, of 8, of none, by a CTA a token and in rings, a skipped request among them."""
    H, G, page = 5, 5, 64
    for tokens in (40, 2600):
        cu = [0, tokens // 3, tokens - 4, tokens]
        new = [b - a for a, b in zip(cu, cu[1:])]
        lengths = [0, 9 + new[1], 100000 + new[2]]
        g = gen(tokens + dim)
        table, pages = ref.table([9 + n for n in new], page, 1600, torch.Generator().manual_seed(1))
        table[2, 1562:1566] = torch.arange(pages, pages + 4, dtype=torch.int32)
        kc, vc = base.pools(g, pages + 4, page, G, dim, dtype, True)
        before = kc.clone(), vc.clone()
        q, k, v = (rand(g, tokens, n, dim, dtype=dtype) for n in (H, G, G))
        freq = rand(g, turned // 2).abs()
        status = word()
        got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32(cu), interleaved=interleaved, amplitude=1.25,
                                device_status=status)
        assert int(status) == 0
        base.rotary_check(q, k, v, freq, list(zip(cu, cu[1:])), lengths, table, kc, vc, interleaved, 1.25, got, before, (0,))


def test_rotary_negative_and_large_frequencies():
    """A frequency of any sign and size counts modulo a turn."""
    dim, page, far = 64, 16, 1000000
    freq = torch.linspace(-40.0, 40.0, dim // 2, device="cuda") + 0.01
    q, k, v = (rand(gen(i), 2, 2, dim) for i in (1, 2, 3))
    table = torch.full((2, far // page + 1), -1, dtype=torch.int32)
    table[0, (far - 1) // page], table[1, 0] = 0, 1
    kc, vc = base.pools(gen(4), 2, page, 2, dim, F32, False)
    before = kc.clone(), vc.clone()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table.cuda(), i32([far, 2]))
    base.rotary_check(q, k, v, freq, [(0, 1), (1, 2)], [far, 2], table.cuda(), kc, vc, False, 1.0, got, before)


@pytest.mark.parametrize("H,G,dim", [(128, 16, 256), (300, 50, 256)])
def test_rotary_long_tokens(H, G, dim):
    """Tokens of which a ring holds few, and of which it holds none (fp32)."""
    T = 2600
    g = gen(1)
    lengths = [T]
    table, pages = ref.table(lengths, 64, 0, torch.Generator().manual_seed(1))
    kc, vc = base.pools(g, pages, 64, G, dim, F32, False)
    before = kc.clone(), vc.clone()
    q, k, v = rand(g, T, H, dim), rand(g, T, G, dim), rand(g, T, G, dim)
    freq, _ = rsm.rotary_frequencies(dim)
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32(lengths), i32([0, T]), interleaved=True)
    base.rotary_check(q, k, v, freq, [(0, T)], lengths, table, kc, vc, True, 1.0, got, before)


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 64), (BF16, 40)])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 3.0])
def test_attention_scales(dtype, dim, scale):
    lengths = [200, 33, 64]
    q, kc, vc, table = base.attention_world(lengths, 2, 4, 2, dim, 16, dtype, False, 21)
    base.attention_check(q, kc, vc, table, lengths, rsm.paged_attention(q, kc, vc, table, i32(lengths), scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("T", [33, 130])
def test_attention_many_new_tokens(T, dtype, dim):
    """Windows whose rows are several units of a key head, from the request's first token on."""
    lengths = [T, 200, T + 1]
    q, kc, vc, table = base.attention_world(lengths, T, 6, 2, dim, 16, dtype, True, T)
    base.attention_check(q, kc, vc, table, lengths, rsm.paged_attention(q, kc, vc, table, i32(lengths)))


def test_attention_does_the_same_twice():
    lengths = [3001, 17, 900, 64]
    q, kc, vc, table = base.attention_world(lengths, 2, 8, 2, 128, 16, BF16, False, 5)
    want = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    for _ in range(20):
        assert torch.equal(rsm.paged_attention(q, kc, vc, table, i32(lengths)), want)


def workspace_bytes(q, kc, table):
    a = hybrid.PagedAttentionArgs()
    a.requests, a.table_width, a.num_pages, a.page_size = *table.shape, *kc.shape[:2]
    a.window, a.num_heads, a.num_kv_heads, a.dim, a.input_dtype = q.shape[1], q.shape[2], kc.shape[2], q.shape[3], rsm.RSM_BF16
    return hybrid._load().rsm_paged_attention_workspace(bytes(a))


def test_attention_workspace():
    """One of the bytes asked for is enough, and what lies behind it stays; less, or off 256 bytes, is refused; a table
    of one tile needs none."""
    lengths = [3001, 17, 900, 64]
    q, kc, vc, table = base.attention_world(lengths, 2, 8, 2, 128, 16, BF16, False, 5)
    want, n = rsm.paged_attention(q, kc, vc, table, i32(lengths)), workspace_bytes(q, kc, table)
    room = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    got = rsm.paged_attention(q, kc, vc, table, i32(lengths), workspace=room[:n])
    assert torch.equal(got, want) and bool((room[n:] == 77).all())
    for bad in (room[:n - 1], room[16:16 + n]):
        with pytest.raises(rsm.ReplaySSMError, match="workspace"):
            rsm.paged_attention(q, kc, vc, table, i32(lengths), workspace=bad)
    assert workspace_bytes(q, kc, table[:, :4]) == 0


def test_attention_lengths_past_the_first_tile_of_many_requests():
    """More requests than a CTA has threads, most of them empty or short, some long: where the work is dealt out."""
    g = torch.Generator().manual_seed(3)
    lengths = [int(n) for n in torch.randint(0, 4, (700,), generator=g)]
    for r, n in ((0, 900), (127, 65), (128, 640), (300, 64), (511, 2000), (699, 130)):
        lengths[r] = n
    q, kc, vc, table = base.attention_world(lengths, 1, 4, 2, 64, 16, BF16, False, 5)
    base.attention_check(q, kc, vc, table, lengths, rsm.paged_attention(q, kc, vc, table, i32(lengths)))


def test_attention_table_rows_apart():
    """A page table that is a slice of a wider one, and K and V that are slices of layers' common pool."""
    lengths = [100, 3, 65]
    q, kc, vc, table = base.attention_world(lengths, 1, 4, 2, 64, 16, BF16, False, 5)
    wide = torch.full((3, 50), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + table.shape[1]] = table
    both = torch.stack([torch.zeros_like(kc), kc, vc], 1)
    got = rsm.paged_attention(q, both[:, 1], both[:, 2], wide[:, 7:7 + table.shape[1]], i32(lengths))
    assert torch.equal(got, rsm.paged_attention(q, kc, vc, table, i32(lengths)))


def laid_out(t, how):
    """The pages' values in another layout."""
    P, page, G, dim = t.shape
    if how == "heads first":
        return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    if how == "padded":  # pages that are no multiple of their rows apart
        room = torch.zeros(P, page * G * dim + 8, dtype=t.dtype, device="cuda")
        room[:, :page * G * dim] = t.reshape(P, -1)
        return room[:, :page * G * dim].unflatten(1, (page, G, dim))
    if how == "joined":
        return torch.stack([t, torch.full_like(t, float("nan"))], 2)[:, :, 0]
    if how == "rows last":  # a page's rows further apart than pages
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    return t


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 256), (BF16, 72), (F32, 64), (F32, 128), (F32, 256)])
@pytest.mark.parametrize("page", [1, 3, 7, 16, 40])
def test_attention_layouts_of_the_pages(page, dtype, dim):
    """Tokens in pages of any size and layout, of one head and several: the same bits as from pages of 16, wherever
    boxes, gathers or single rows are loaded; what lies beside them is not a number, pages out of range are not seen."""
    lengths, T = [700, 33, 0, 5, 64, 129], 2
    for G in (1, 3):
        q, kc, vc, table = base.attention_world(lengths, T, 4 * G, G, dim, 16, dtype, False, 31 + G)
        want = rsm.paged_attention(q, kc, vc, table, i32(lengths))
        width = -(-700 // page)
        order = torch.randperm(len(lengths) * width, generator=torch.Generator().manual_seed(3)).to("cuda")
        other = order.view(len(lengths), width).int()
        pools = [torch.full((len(order), page, G, dim), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
        for b, n in enumerate(lengths):
            at = torch.arange(n, device="cuda")
            for pool, c in zip(pools, (kc, vc)):
                pool[other[b, at // page].long(), at % page] = c[table[b, at // 16].long(), at % 16]
        for hk, hv in (("", ""), ("heads first", "heads first"), ("padded", "padded"), ("joined", "joined"), ("", "heads first"),
                       ("rows last", "rows last"), ("padded", "joined")):
            k, v = laid_out(pools[0], hk), laid_out(pools[1], hv)
            status = word()
            got = rsm.paged_attention(q, k, v, other, i32(lengths), device_status=status)
            assert torch.equal(got, want) and int(status) == 0, (G, hk, hv)
        bad = other.clone()
        bad[0, width // 2] = len(order)
        bad[4, 0] = -1
        got = rsm.paged_attention(q, pools[0], pools[1], bad, i32(lengths), device_status=status)
        assert int(status) == 128 and torch.equal(got[[1, 2, 3, 5]], want[[1, 2, 3, 5]]) and bool(torch.isfinite(got).all())
        live = torch.ones(700, dtype=torch.bool)
        live[width // 2 * page:(width // 2 + 1) * page] = False
        at = torch.arange(700, device="cuda")
        for h in range(4 * G):
            s = (pools[0][other[0, at // page].long(), at % page, h // 4].double() @ q[0, :, h].double().T) * dim ** -0.5
            for t in range(T):
                see = live.to("cuda") & (at <= 700 - T + t)
                w = torch.softmax(s[:, t].masked_fill(~see, -torch.inf), 0)
                vals = vc[table[0, at // 16].long(), at % 16, h // 4].double()
                y, m = w @ vals, w @ vals.abs()
                bound = (2.0 ** -8 * (y.abs() + m) if dtype == BF16 else 0 * m) + 1e-4 * (1 + m)
                assert bool(((got[0, t, h].double() - y).abs() <= bound).all())


@pytest.mark.parametrize("page", [16, 8])
def test_attention_pages_past_2_31_values(page):
    """Pages whose offsets pass 32 bits, by boxes and by rows."""
    G, dim, n = 16, 128, 300
    pages = 2 ** 31 // (page * G * dim) + 40
    kc, vc = (torch.zeros(pages, page, G, dim, device="cuda", dtype=BF16) for _ in range(2))
    need = -(-n // page)
    at = torch.arange(pages - need, pages, device="cuda")
    kc[at], vc[at] = rand(gen(1), need, page, G, dim, dtype=BF16), rand(gen(2), need, page, G, dim, dtype=BF16)
    q = rand(gen(3), 1, 1, 32, dim, dtype=BF16, scale=2.0)
    got = rsm.paged_attention(q, kc, vc, at[None].int(), i32([n]))
    few = torch.arange(need, device="cuda", dtype=torch.int32)[None]
    assert torch.equal(got, rsm.paged_attention(q, kc[at].clone(), vc[at].clone(), few, i32([n])))
    freq, _ = rsm.rotary_frequencies(dim)
    new = [rand(gen(i), 1, 1, h, dim, dtype=BF16) for i, h in ((5, 32), (6, G), (7, G))]
    k2, v2 = kc[at].clone(), vc[at].clone()
    a = rsm.rotary_append(*new, freq, kc, vc, at[None].int(), i32([n]))
    assert torch.equal(a, rsm.rotary_append(*new, freq, k2, v2, few, i32([n])))
    assert torch.equal(kc[at], k2) and torch.equal(vc[at], v2)


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 64), (BF16, 40)])
def test_attention_scores_that_are_infinite(dtype, dim):
    """A key that makes a score -infinity takes no weight; one that makes it +infinity makes the row NaN, as the
    quotient of infinities is; other heads and requests are as ever."""
    lengths = [70, 70]
    q, kc, vc, table = base.attention_world(lengths, 1, 4, 4, dim, 16, dtype, False, 5)
    q = q.abs() + 0.1
    want = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    k2 = kc.clone()
    k2[table[0, 1].item(), 3, 1] = -float("inf")
    got = rsm.paged_attention(q, k2, vc, table, i32(lengths))
    lone = [i for i in range(70) if i != 19]
    p = torch.tensor(lone, device="cuda")
    k = kc[table[0, p // 16].long(), p % 16, 1].double()
    w = torch.softmax(k @ q[0, 0, 1].double() * dim ** -0.5, 0)
    v = vc[table[0, p // 16].long(), p % 16, 1].double()
    m = w @ v.abs()
    top = (k.abs() @ q[0, 0, 1].double().abs()).max() * dim ** -0.5
    close(got[0, 0, 1], w @ v, base.attention_bound(w @ v, m, top, dim, 70, dtype))
    k2[table[0, 1].item(), 3, 1] = float("inf")
    odd = rsm.paged_attention(q, k2, vc, table, i32(lengths))
    assert bool(odd[0, 0, 1].isnan().all())
    for y in (got, odd):
        y[0, 0, 1] = want[0, 0, 1]
        assert torch.equal(y, want)


def test_nothing_to_do():
    z = lambda *s, t=BF16: torch.zeros(s, device="cuda", dtype=t)  # noqa: E731
    w, none = z(8, 4, t=F32), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert rsm.causal_conv(z(0, 8), w, i32([0])).shape == (0, 8)
    assert rsm.causal_conv(z(0, 8), w, i32([0, 0]), None, z(1, 3, 8), i32([0])).shape == (0, 8)
    assert rsm.causal_conv_step(z(0, 8), w, z(1, 4, 8), none, none).shape == (0, 8)
    kc, table = z(2, 4, 1, 8), torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    assert rsm.rotary_append(z(0, 2, 8), z(0, 1, 8), z(0, 1, 8), z(4, t=F32), kc, kc.clone(), table, none).shape == (0, 2, 8)
    assert rsm.paged_attention(z(0, 2, 8), kc, kc, table, none).shape == (0, 2, 8)
    y = rsm.paged_attention(torch.ones(2, 2, 64, device="cuda"), z(0, 4, 1, 64, t=F32), z(0, 4, 1, 64, t=F32),
                            torch.zeros(2, 0, dtype=torch.int32, device="cuda"), i32([0, 0]))
    assert bool((y == 0).all())
    rsm.copy_pages(rsm.pointer_table([kc]), rsm.stride_table([kc]), none, none, dtype=BF16, page_elements=32, num_pages=2)


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 64), (F32, 128), (BF16, 40)])
@pytest.mark.parametrize("inf", [float("inf"), -float("inf")])
def test_attention_values_that_are_infinite(dtype, dim, inf):
    """An infinite value that a row sees makes its column infinite, and no other."""
    lengths = [150, 70]
    q, kc, vc, table = base.attention_world(lengths, 3, 4, 2, dim, 16, dtype, False, 5)
    want = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    v2 = vc.clone()
    v2[table[0, 2].item(), 3, 1, 7] = inf      # token 35 of request 0, seen by all its rows
    v2[table[1, 4].item(), 4, 0, 3] = inf      # token 68 of request 1: seen by its last two
    got = rsm.paged_attention(q, kc, v2, table, i32(lengths))
    assert bool((got[0, :, 2:, 7] == inf).all()) and bool((got[1, 1:, :2, 3] == inf).all())
    got[0, :, 2:, 7], got[1, 1:, :2, 3] = want[0, :, 2:, 7], want[1, 1:, :2, 3]
    assert torch.equal(got, want)
