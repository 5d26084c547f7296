"""The layer operators on a GPU against their definition in 64 bits.

Error bounds, per element.  u = 2^-8 is bf16's half unit (8 significant bits), M the sum of the
absolute values of the terms an element is made of (computed alongside the
reference).  With bf16 inputs a term of an output may pass one rounding to bf16
on its way (the weight of a token pair, or the state), fp32 accumulation adds
at most a few hundred roundings of 2^-24, and the output is rounded once:
  |y - exact| <= u |exact| + (u + 2^-15) M.
A state's terms keep 16 bits or more for fp32 and fp16 states and 8 for bf16
states, plus the rounding to the stored type.  With fp32 inputs every step
multiplies by exp(dt A): a rounded product, an exponential within 2 units and
an fma, 1.5 2^-22 a token, so L tokens are within L 2^-21 M.
"""
import pytest

torch = pytest.importorskip("torch")

import block_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 1e-38, F16: 2.0 ** -25, F32: 1e-38}  # absolute, for values below the normal range


def close(got, want, rel, sums, by_sums, what):
    err = (got.double() - want).abs()
    bound = rel * want.abs() + by_sums * sums + TINY[got.dtype]
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float((err / bound).max()):.3g}"


def y_terms(dtype, tokens):
    return 2.0 ** -8 + 2.0 ** -15 if dtype == BF16 else (tokens + 64) * 2.0 ** -21


def state_terms(inputs, state, tokens):
    if inputs == BF16:
        return 2.0 ** -8 + 2.0 ** -15 if state == BF16 else 2.0 ** -15
    return (tokens + 64) * 2.0 ** -21


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tokens(lead, H, G, dim, N, dtype, seed, sliced=0, strong=False):
    """x, dt, A, B, C, D; sliced: x, B, C are slices of one tensor starting at that element."""
    g = gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if sliced:
        w = H * dim + 2 * G * N
        t = rn(*lead, w + sliced + 7).to(dtype)[..., sliced:sliced + w]
        x, B, C = t.split([H * dim, G * N, G * N], dim=-1)
        x, B, C = x.unflatten(-1, (H, dim)), B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N))
    else:
        x, B, C = rn(*lead, H, dim).to(dtype), rn(*lead, G, N).to(dtype), rn(*lead, G, N).to(dtype)
    dt = 0.001 + (3.0 if strong else 0.1) * torch.rand((*lead, H), generator=g, device="cuda")
    A = -(0.5 + 1.5 * torch.rand(H, generator=g, device="cuda")) * (16.0 if strong else 1.0)
    return x, dt, A, B, C, rn(H)


def pool(slots, H, dim, N, dtype, seed):
    return torch.randn((slots, H, dim, N), generator=gen(seed), device="cuda", dtype=F32).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_prefill(lens, H, G, dim, N, inputs, state_dtype, initial=True, skip=True, sliced=0, strong=False, seed=0):
    T, S = sum(lens), len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x, dt, A, B, C, D = tokens((T,), H, G, dim, N, inputs, seed, sliced, strong)
    D = D if skip else None
    st = pool(2 * S + 1, H, dim, N, state_dtype, seed + 1)
    before = st.clone()
    ini, fin = list(range(S)), list(range(2 * S - 1, S - 1, -1))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = rsm.ssm_prefill(x, dt, A, B, C, i32(cu), st, initial_slots=i32(ini) if initial else None,
                        final_slots=i32(fin), D=D, device_status=status)
    wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, cu, before, ini if initial else None, D)
    L = max(lens)
    assert y.shape == x.shape and y.dtype == inputs and int(status) == 0
    close(y, wy, HALF_UNIT[inputs], wm, y_terms(inputs, L), "y")
    close(st[fin], ws, HALF_UNIT[state_dtype], wsm, state_terms(inputs, state_dtype, L), "state")
    keep = [i for i in range(2 * S + 1) if i not in fin]
    assert torch.equal(st[keep], before[keep]), "slots that are not final slots changed"


LENGTHS = [[1], [2, 1, 3], [31, 32, 33], [63, 64, 65], [127, 128, 129], [255, 256, 257, 1], [0, 5, 0, 130, 0], [700]]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("state", [F32, BF16, F16])
def test_prefill_lengths(lens, state):
    check_prefill(lens, 8, 2, 64, 128, BF16, state, seed=len(lens))


@pytest.mark.parametrize("H,G", [(1, 1), (2, 1), (3, 1), (4, 4), (6, 2), (9, 3), (80, 1), (20, 4)])
def test_prefill_heads(H, G):
    check_prefill([37, 150], H, G, 64, 128, BF16, F32, seed=H)


@pytest.mark.parametrize("dim,N", [(16, 16), (64, 64), (64, 128)])
@pytest.mark.parametrize("inputs", [BF16, F32])
@pytest.mark.parametrize("initial,skip", [(True, False), (False, True)])
def test_prefill_sizes_and_types(dim, N, inputs, initial, skip):
    check_prefill([5, 70, 200], 6, 2, dim, N, inputs, F32, initial=initial, skip=skip, seed=dim + N)


@pytest.mark.parametrize("sliced", [1, 4, 8, 64])
def test_prefill_slices_of_a_projection(sliced):
    check_prefill([40, 129], 4, 2, 64, 128, BF16, F32, sliced=sliced, seed=sliced)


def test_prefill_strong_decay():
    """Steps that decay the state to nothing within a few tokens, and within one."""
    check_prefill([300, 77], 4, 1, 64, 128, BF16, F32, strong=True, seed=3)


@pytest.mark.parametrize("state", [F32, BF16])
def test_prefill_long_sequence_of_few_heads(state):
    check_prefill([3001], 2, 1, 64, 128, BF16, state, seed=11)
    check_prefill([1500, 9, 2200], 3, 1, 64, 128, BF16, state, seed=12, initial=False)


def test_prefill_repeats_bit_for_bit():
    x, dt, A, B, C, D = tokens((900,), 4, 1, 64, 128, BF16, 5)
    cu = i32([0, 900])
    outs = []
    for _ in range(3):
        st = torch.zeros(1, 4, 64, 128, device="cuda")
        outs.append((rsm.ssm_prefill(x, dt, A, B, C, cu, st, final_slots=i32([0]), D=D), st))
    for y, st in outs[1:]:
        assert torch.equal(y, outs[0][0]) and torch.equal(st, outs[0][1])


def test_prefill_pieces_equal_the_whole():
    """A prompt in two calls, the state carried in its slot in place, against the prompt in one."""
    x, dt, A, B, C, D = tokens((333,), 4, 2, 64, 128, BF16, 6)
    st = torch.zeros(1, 4, 64, 128, device="cuda")
    a = rsm.ssm_prefill(x[:200], dt[:200], A, B[:200], C[:200], i32([0, 200]), st, final_slots=i32([0]), D=D)
    b = rsm.ssm_prefill(x[200:], dt[200:], A, B[200:], C[200:], i32([0, 133]), st, initial_slots=i32([0]),
                        final_slots=i32([0]), D=D)
    wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, [0, 333], st, None, D)
    close(torch.cat([a, b]), wy, 2.0 ** -8, wm, y_terms(BF16, 333), "y")
    close(st, ws, 2.0 ** -24, wsm, 2.0 ** -15, "state")


def test_prefill_pads_bad_slots_and_bad_sequences():
    x, dt, A, B, C, D = tokens((60,), 4, 2, 64, 128, BF16, 7)
    st = pool(3, 4, 64, 128, F32, 8)
    before = st.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = rsm.ssm_prefill(x, dt, A, B, C, i32([0, 20, 60]), st, initial_slots=i32([-1, 1]), final_slots=i32([2, -1]), D=D,
                        device_status=status)
    wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, [0, 20, 60], before, [-1, 1], D)
    assert int(status) == 0
    close(y, wy, 2.0 ** -8, wm, y_terms(BF16, 60), "y")
    close(st[2:3], ws[:1], 2.0 ** -24, wsm[:1], 2.0 ** -15, "state")
    assert torch.equal(st[:2], before[:2])
    # slots out of range: as pads, and flagged
    y2 = rsm.ssm_prefill(x, dt, A, B, C, i32([0, 20, 60]), st, initial_slots=i32([7, 1]), final_slots=i32([2, -9]), D=D,
                         device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_slot"] and torch.equal(y2, y)
    # a sequence that ends past the tokens or before its start is skipped
    status.zero_()
    out = torch.full_like(x, 3.0)
    rsm.ssm_prefill(x, dt, A, B, C, i32([0, 20, 61]), st, D=D, out=out, device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_sequence"]
    assert (out[20:] == 3.0).all()
    wy2 = ref.prefill(x, dt, A, B, C, [0, 20], before, None, D)
    close(out[:20], wy2[0][:20], 2.0 ** -8, wy2[1][:20], y_terms(BF16, 20), "first sequence")


def test_prefill_no_tokens_keeps_the_state():
    x, dt, A, B, C, D = tokens((0,), 4, 2, 64, 128, BF16, 7)
    st = pool(3, 4, 64, 128, BF16, 8)
    before = st.clone()
    y = rsm.ssm_prefill(x, dt, A, B, C, i32([0, 0, 0]), st, initial_slots=i32([0, -1]), final_slots=i32([1, 2]), D=D)
    assert y.numel() == 0 and torch.equal(st[0], before[0]) and torch.equal(st[1], before[0]) and not st[2].any()


def test_prefill_non_finite_values_stay_in_their_sequence():
    """A neighbour's NaN and infinity, right after a ragged end, reach nothing."""
    for bad in (float("nan"), float("inf")):
        x, dt, A, B, C, D = tokens((200,), 4, 2, 64, 128, BF16, 9)
        clean = rsm.ssm_prefill(x, dt, A, B, C, i32([0, 90, 200]), D=D)
        x2, B2, C2 = x.clone(), B.clone(), C.clone()
        x2[90:], B2[90:], C2[90:] = bad, bad, bad
        st = torch.zeros(2, 4, 64, 128, device="cuda")
        y = rsm.ssm_prefill(x2, dt, A, B2, C2, i32([0, 90, 200]), st, final_slots=i32([0, 1]), D=D)
        assert torch.equal(y[:90], clean[:90]) and torch.isfinite(st[0]).all()


def test_prefill_on_another_stream():
    x, dt, A, B, C, D = tokens((500,), 8, 2, 64, 128, BF16, 10)
    want = rsm.ssm_prefill(x, dt, A, B, C, i32([0, 500]), D=D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rsm.ssm_prefill(x, dt, A, B, C, i32([0, 500]), D=D, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


# ----------------------------------------------------------------------------
# running requests
# ----------------------------------------------------------------------------

def check_step(b, T, H, G, dim, N, inputs, state_dtype, in_place, pads=(), sliced=0, seed=0, skip=True, strong=False):
    x, dt, A, B, C, D = tokens((b, T), H, G, dim, N, inputs, seed, sliced, strong)
    D = D if skip else None
    st = pool(2 * b + 1, H, dim, N, state_dtype, seed + 1)
    before = st.clone()
    src = [i if i not in pads else -1 for i in range(b)]
    dst = src if in_place else [2 * b - 1 - i for i in range(b)]
    y = rsm.ssm_step(st, i32(src), x, dt, A, B, C, dst_slots=None if in_place else i32(dst), D=D)
    Dw = torch.zeros(H, device="cuda") if D is None else D
    written = set()
    for i in range(b):
        if src[i] < 0:
            assert not y[i].any()
            continue
        S = ref.f64(before[src[i]])
        wy, wm, ws, wsm = ref.run_tokens(S, S.abs(), *(ref.f64(t) for t in (x[i], dt[i], A, B[i], C[i], Dw)))
        close(y[i], wy, HALF_UNIT[inputs], wm, y_terms(inputs, T), f"y of request {i}")
        close(st[dst[i]], ws, HALF_UNIT[state_dtype], wsm, state_terms(inputs, state_dtype, T), f"state of request {i}")
        written.add(dst[i])
    keep = [i for i in range(2 * b + 1) if i not in written]
    assert torch.equal(st[keep], before[keep])


@pytest.mark.parametrize("state", [F32, BF16, F16])
@pytest.mark.parametrize("T", [1, 2, 3, 8])
@pytest.mark.parametrize("in_place", [True, False])
def test_step(state, T, in_place):
    check_step(5, T, 8, 2, 64, 128, BF16, state, in_place, pads=(1,), seed=T)


@pytest.mark.parametrize("dim,N", [(16, 16), (64, 64), (64, 128)])
@pytest.mark.parametrize("inputs", [BF16, F32])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 3), (9, 3), (80, 1)])
def test_step_sizes(dim, N, inputs, H, G):
    check_step(2, 1, H, G, dim, N, inputs, F32, True, seed=H, skip=False)
    check_step(1, 5, H, G, dim, N, inputs, F16, False, sliced=3, seed=H)


def test_step_strong_decay_and_long_windows():
    check_step(2, 70, 4, 1, 64, 128, BF16, F32, True, seed=2)
    check_step(2, 4, 4, 1, 64, 128, BF16, F32, True, seed=2, strong=True)


def test_step_without_the_window_dimension():
    x, dt, A, B, C, D = tokens((3,), 4, 2, 64, 128, BF16, 4)
    st = pool(3, 4, 64, 128, BF16, 5)
    st2 = st.clone()
    y = rsm.ssm_step(st, i32([0, 1, 2]), x, dt, A, B, C, D=D)
    y2 = rsm.ssm_step(st2, i32([0, 1, 2]), x[:, None], dt[:, None], A, B[:, None], C[:, None], D=D)
    assert y.shape == x.shape and torch.equal(y, y2[:, 0]) and torch.equal(st, st2)


def test_step_flags_bad_slots():
    x, dt, A, B, C, D = tokens((3, 1), 4, 2, 64, 128, BF16, 4)
    st = pool(3, 4, 64, 128, BF16, 5)
    before = st.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = rsm.ssm_step(st, i32([0, 3, -5]), x, dt, A, B, C, dst_slots=i32([-1, 1, 2]), D=D, device_status=status)
    assert int(status) == rsm.STATUS_BITS["bad_slot"]
    assert y[0].any() and not y[1:].any() and torch.equal(st, before)


# ----------------------------------------------------------------------------
# ring decode
# ----------------------------------------------------------------------------

def check_decode(b, T, R, H, G, dim, N, inputs, state, lens=None, pads=(), seed=0, skip=True, sliced=0):
    x, dt, A, B, C, D = tokens((b, T), H, G, dim, N, inputs, seed, sliced)
    D = D if skip else None
    S = b + 1
    xc, dtc, _, Bc, _, _ = tokens((S, R), H, G, dim, N, inputs, seed + 50)
    g = torch.Generator().manual_seed(seed)
    scale = None
    if state in (torch.int8, torch.float8_e4m3fn):
        st = torch.randint(-127, 128, (S, H, dim, N), generator=gen(seed), device="cuda", dtype=torch.int8)
        if state != torch.int8:
            st = (st.to(F16) * 3.5).to(state)
        scale = 0.01 + 0.05 * torch.rand((S, H, dim), generator=gen(seed + 1), device="cuda")
        values = st.double() * scale.double()[..., None]
    else:
        st = pool(S, H, dim, N, state, seed + 1)
        values = st.double()
    slots = (torch.randperm(b, generator=g) + 1).tolist()
    slots = [s if i not in pads else -1 for i, s in enumerate(slots)]
    start = torch.randint(0, R, (b,), generator=g).tolist()
    have = lens or torch.randint(0, R - T + 1, (b,), generator=g).tolist()
    caches = [t.clone() for t in (xc, Bc, dtc)]
    raw = st.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = rsm.replayssm_decode(st, i32(slots), *caches, i32(start), i32(have), x, dt, A, B, C, state_scale=scale, D=D,
                             device_status=status)
    assert int(status) == 0
    want = [t.clone() for t in (xc, Bc, dtc)]
    for i in range(b):
        s = slots[i]
        if s < 0:
            assert not y[i].any()
            continue
        rows = [(start[i] + k) % R for k in range(have[i])]
        cat = lambda c, n: torch.cat([ref.f64(c[s, rows]), ref.f64(n[i])])  # noqa: E731
        Cs = torch.cat([torch.zeros(have[i], G, N, dtype=torch.float64, device="cuda"), ref.f64(C[i])])
        Dw = torch.zeros(H, device="cuda") if D is None else D
        wy, wm, _, _ = ref.run_tokens(values[s], values[s].abs(), cat(xc, x), cat(dtc, dt), ref.f64(A), cat(Bc, B), Cs,
                                      ref.f64(Dw))
        close(y[i], wy[have[i]:], HALF_UNIT[inputs], wm[have[i]:], y_terms(inputs, R), f"y of request {i}")
        for k in range(T):
            row = (start[i] + have[i] + k) % R
            for w, n in zip(want, (x, B, dt)):
                w[s, row] = n[i, k]
    for w, c in zip(want, caches):
        assert torch.equal(w, c), "ring rows"
    assert torch.equal(st.view(torch.uint8), raw.view(torch.uint8))


STATES = [F32, BF16, F16, torch.int8, torch.float8_e4m3fn]


@pytest.mark.parametrize("state", STATES, ids=str)
@pytest.mark.parametrize("T", [1, 2, 4, 5, 8])
def test_decode(state, T):
    check_decode(6, T, 16, 8, 2, 64, 128, BF16, state, pads=(2,), seed=T)


@pytest.mark.parametrize("inputs", [BF16, F32])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 3), (9, 3), (80, 1), (34, 2)])
def test_decode_heads(inputs, H, G):
    check_decode(2, 1, 8, H, G, 64, 128, inputs, BF16, seed=H)
    check_decode(2, 3, 8, H, G, 64, 128, inputs, torch.int8, seed=H, skip=False, sliced=5)


@pytest.mark.parametrize("dim,N", [(16, 16), (64, 64)])
@pytest.mark.parametrize("inputs", [BF16, F32])
def test_decode_sizes(dim, N, inputs):
    check_decode(3, 2, 8, 4, 2, dim, N, inputs, F32, seed=dim)


def test_decode_empty_full_and_long_rings():
    check_decode(3, 1, 8, 4, 2, 64, 128, BF16, BF16, lens=[0, 7, 3])
    check_decode(2, 8, 8, 4, 2, 64, 128, BF16, BF16, lens=[0, 0])
    check_decode(2, 16, 64, 4, 2, 64, 128, BF16, F16, lens=[48, 1])
    check_decode(2, 64, 64, 2, 1, 64, 128, BF16, F32, lens=[0, 0])
    check_decode(2, 3, 100, 2, 1, 64, 128, BF16, F32, lens=[61, 60])


def test_decode_flags_bad_metadata():
    x, dt, A, B, C, D = tokens((4, 1), 4, 2, 64, 128, BF16, 4)
    xc, dtc, _, Bc, _, _ = tokens((4, 8), 4, 2, 64, 128, BF16, 5)
    st = pool(4, 4, 64, 128, BF16, 5)
    for name, slots, start, have in (("bad_slot", [0, 4, 2, 3], [0, 0, 0, 0], [0, 0, 0, 0]),
                                     ("bad_ring_start", [0, 1, 2, 3], [0, 8, 0, 0], [0, 0, 0, 0]),
                                     ("bad_prefix_len", [0, 1, 2, 3], [0, 0, 0, 0], [0, 8, 0, 0]),
                                     ("bad_prefix_len", [0, 1, 2, 3], [0, 0, 0, 0], [0, -1, 0, 0])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        caches = [t.clone() for t in (xc, Bc, dtc)]
        y = rsm.replayssm_decode(st, i32(slots), *caches, i32(start), i32(have), x, dt, A, B, C, D=D,
                                 device_status=status)
        assert int(status) == rsm.STATUS_BITS[name]
        assert not y[1].any() and y[0].any() and y[2].any()
        assert torch.equal(caches[0][1], xc[1]) and torch.equal(caches[1][1], Bc[1]) and torch.equal(caches[2][1], dtc[1])


def test_decode_reads_slots_past_32_bit_offsets():
    """A pool whose last slot starts past 2^31 elements (4.3 GB of bf16)."""
    H = 4
    per = H * 64 * 128
    n = (1 << 31) // per + 2
    st = torch.zeros((n, H, 64, 128), dtype=BF16, device="cuda")
    x, dt, A, B, C, D = tokens((1, 1), H, 1, 64, 128, BF16, 4)
    st[n - 1] = pool(1, H, 64, 128, BF16, 3)[0]
    S = ref.f64(st[n - 1])
    wy, wm, ws, wsm = ref.run_tokens(S, S.abs(), *(ref.f64(t) for t in (x[0], dt[0], A, B[0], C[0], D)))
    y = rsm.ssm_step(st, i32([n - 1]), x, dt, A, B, C, dst_slots=i32([n - 2]), D=D)
    close(y[0], wy, 2.0 ** -8, wm, y_terms(BF16, 1), "y")
    close(st[n - 2], ws, 2.0 ** -8, wsm, state_terms(BF16, BF16, 1), "state")


def test_decode_then_materialize_equals_step():
    """Four tokens decoded onto the ring, then committed by replayssm_materialize, against ssm_step in place."""
    H, G, b, R = 8, 2, 3, 8
    x, dt, A, B, C, D = tokens((b, 4), H, G, 64, 128, BF16, 14)
    st = pool(2 * b, H, 64, 128, F32, 15)
    st2 = st.clone()
    caches = [torch.zeros(2 * b, R, H, 64, dtype=BF16, device="cuda"), torch.zeros(2 * b, R, G, 128, dtype=BF16, device="cuda"),
              torch.zeros(2 * b, R, H, device="cuda")]
    slots, start, have = i32([0, 1, 2]), i32([5, 0, 7]), i32([0, 0, 0])
    ys = []
    for t in range(4):
        ys.append(rsm.replayssm_decode(st, slots, *caches, start, have, x[:, t], dt[:, t], A, B[:, t], C[:, t], D=D))
        have += 1
    tab, strd = rsm.pointer_table, rsm.stride_table
    rsm.replayssm_materialize(tab([st]), strd([st]), tab([caches[0]]), strd([caches[0]]), tab([caches[1]]),
                              strd([caches[1]]), tab([caches[2]]), strd([caches[2]]), tab([A]), None, None,
                              slots[None].contiguous(), i32([[3, 4, 5]]), start, have, i32([0, 1, 2]),
                              state_dtype=F32, input_dtype=BF16, matrixA_dtype=F32, dim=64, dstate=128, num_heads=H,
                              heads_per_group=H // G, max_window=R, ring_buffer_len=R)
    y2 = rsm.ssm_step(st2, slots, x, dt, A, B, C, D=D)
    for i in range(b):
        S = ref.f64(st[i])
        wy, wm, ws, wsm = ref.run_tokens(S, S.abs(), *(ref.f64(t) for t in (x[i], dt[i], A, B[i], C[i], D)))
        close(torch.stack(ys, 1)[i], wy, 2.0 ** -8, wm, y_terms(BF16, R), "ring outputs")
        close(y2[i], wy, 2.0 ** -8, wm, y_terms(BF16, R), "step outputs")
        close(st[3 + i], ws, 2.0 ** -24, wsm, 2.0 ** -15, "materialized state")
        close(st2[i], ws, 2.0 ** -24, wsm, 2.0 ** -15, "stepped state")


# ----------------------------------------------------------------------------
# norms.  With r the group's values: each is within 4 units of fp32 (silu: an
# exponential within 2 units, a sum, a quotient), their mean square within
# 2^-20, so the norm before its last rounding within 2^-18 relative.
# ----------------------------------------------------------------------------

NORM_REL = 2.0 ** -18


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (2, 8), (5, 1000), (4, 1023), (2, 5120), (3, 4096), (2, 20000),
                                      (300, 256)])
@pytest.mark.parametrize("inputs", [BF16, F32])
@pytest.mark.parametrize("residual", [BF16, F32])
def test_add_rms_norm(rows, dim, inputs, residual):
    g = gen(dim)
    x = torch.randn((rows, dim), generator=g, device="cuda").to(inputs)
    r = (3 * torch.randn((rows, dim), generator=g, device="cuda")).to(residual)
    w = 0.5 + torch.rand(dim, generator=g, device="cuda")
    y, q = rsm.add_rms_norm(x, r, w, residual_scale=0.7, eps=1e-5)
    s = torch.tensor(0.7, dtype=F32).double().item()
    v = ref.f64(r) + s * ref.f64(x)
    want = ref.rms(v, w.double(), dim, 1e-5)
    size = (ref.f64(r).abs() + s * ref.f64(x).abs())
    close(q, v, HALF_UNIT[residual], size, 2.0 ** -23, "residual")
    close(y, want, HALF_UNIT[inputs] + NORM_REL, ref.rms(v, w.double(), dim, 1e-5).abs() * size / v.abs().clamp(min=1e-30),
          2.0 ** -22, "norm")
    # in place
    x2, r2 = x.clone(), r.clone()
    y2, q2 = rsm.add_rms_norm(x2, r2, w, residual_scale=0.7, eps=1e-5, out=x2, residual_out=r2)
    assert y2 is x2 and q2 is r2 and torch.equal(x2, y) and torch.equal(r2, q)


@pytest.mark.parametrize("rows,dim,group", [(1, 1, 1), (3, 14, 7), (2, 64, 8), (5, 1000, 200), (2, 5120, 5120),
                                            (3, 8192, 1024), (2, 40000, 20000), (300, 512, 64), (7, 4096, 2048)])
@pytest.mark.parametrize("inputs", [BF16, F32])
@pytest.mark.parametrize("first", [False, True])
def test_gated_rms_norm(rows, dim, group, inputs, first):
    g = gen(dim + group)
    x = torch.randn((rows, dim), generator=g, device="cuda").to(inputs)
    z = (4 * torch.randn((rows, dim), generator=g, device="cuda")).to(inputs)
    w = 0.5 + torch.rand(dim, generator=g, device="cuda")
    y = rsm.gated_rms_norm(x, z, w, group_size=group, eps=1e-5, norm_before_gate=first)
    gate = ref.silu(ref.f64(z))
    want = ref.rms(ref.f64(x), w.double(), group, 1e-5) * gate if first else ref.rms(ref.f64(x) * gate, w.double(), group, 1e-5)
    close(y, want, HALF_UNIT[inputs] + NORM_REL, want, 0.0, "norm")
    x2 = x.clone()
    assert torch.equal(rsm.gated_rms_norm(x2, z, w, group_size=group, eps=1e-5, norm_before_gate=first, out=x2), y)


@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_norms_of_slices(offset):
    """Rows that are slices of wider ones, at aligned and odd starts, and a leading dimension more."""
    g = gen(offset)
    t = torch.randn((6, 3, 2100), generator=g, device="cuda").to(BF16)
    x, z = t[..., offset:offset + 1000], t[..., offset + 1003:offset + 2003]
    w = 0.5 + torch.rand(1000, generator=g, device="cuda")
    y = rsm.gated_rms_norm(x, z, w, group_size=200)
    assert torch.equal(y, rsm.gated_rms_norm(x.contiguous(), z.contiguous(), w, group_size=200))
    y, r = rsm.add_rms_norm(x, z, w)
    y2, r2 = rsm.add_rms_norm(x.contiguous(), z.contiguous(), w)
    assert torch.equal(y, y2) and torch.equal(r, r2)


def test_norms_of_extreme_rows():
    """Rows of zeros, of one infinity, and gates far out on either side."""
    w = torch.ones(512, device="cuda")
    x = torch.zeros(3, 512, device="cuda")
    y, r = rsm.add_rms_norm(x, x, w)
    assert not y.any() and not r.any()
    x = torch.randn((2, 512), generator=gen(1), device="cuda")
    x[0, 5] = float("inf")
    y, _ = rsm.add_rms_norm(x, torch.zeros_like(x), w)
    assert torch.isnan(y[0, 5]) and torch.isfinite(y[1]).all() and not y[0, :5].any()
    z = torch.tensor([-200.0, -90.0, 90.0, 200.0], device="cuda").repeat(2, 128)
    x = torch.ones(2, 512, device="cuda")
    y = rsm.gated_rms_norm(x, z, w, eps=1e-5)
    assert torch.isfinite(y).all() and (y[:, 0::4] == 0).all() and (y[:, 3::4] > 0).all()


def test_norms_of_no_rows():
    x = torch.zeros(0, 64, device="cuda", dtype=BF16)
    w = torch.ones(64, device="cuda")
    assert rsm.gated_rms_norm(x, x, w).shape == (0, 64)
    assert rsm.add_rms_norm(x, x, w)[1].shape == (0, 64)
