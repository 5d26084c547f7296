"""The layer operators where a call's metadata, magnitudes or callers are unusual.  Bounds and references are
test_block_ops_gpu's, or stated at the test."""
import threading

import pytest

torch = pytest.importorskip("torch")

import block_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402
import test_block_ops_gpu as base  # noqa: E402
from mamba_replayssm_state_gb300 import block  # noqa: E402
from test_block_ops_gpu import BF16, F16, F32, i32  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def prefill_workspace(T, seqs, H, G):
    """Bytes that a bf16 call of this size needs; 0 where it is not cut into segments."""
    a = block.SsmPrefillArgs()
    a.tokens, a.num_seqs, a.num_heads, a.num_groups, a.dim, a.dstate = T, seqs, H, G, 64, 128
    a.state_dtype, a.input_dtype = rsm.RSM_F32, rsm.RSM_BF16
    return block._load().rsm_ssm_prefill_workspace(bytes(a))


@pytest.mark.parametrize("case", ["cut", "longest first", "many", "one by one"])
def test_prefill_sequences_that_start_over_are_skipped(case):
    """cu_seqlens that goes back and starts over: what would lie over an earlier sequence is skipped and flagged,
    whichever way the call runs, and nothing is written but the first sequence's outputs, its state and, within the
    bytes asked for, the workspace."""
    H, G = 2, 1
    T, inputs = {"cut": (5000, BF16), "longest first": (300, BF16), "many": (300, BF16), "one by one": (150, F32)}[case]
    cu = [0, T, 0, T] if case != "many" else [0, T] + [0, T] * 20
    S = len(cu) - 1
    x, dt, A, B, C, D = base.tokens((T,), H, G, 64, 128, inputs, 3)
    st = base.pool(S + 1, H, 64, 128, F32, 4)
    first = base.pool(S + 1, H, 64, 128, F32, 4)
    want = rsm.ssm_prefill(x, dt, A, B, C, i32([0, T]), first, initial_slots=i32([0]), final_slots=i32([1]), D=D)
    before, status = st.clone(), word()
    size = prefill_workspace(T, S, H, G) if inputs == BF16 else 0
    assert (size > 0) == (case == "cut")
    workspace = torch.full((size + (64 << 20),), 77, dtype=torch.uint8, device="cuda")
    workspace, beyond = workspace[:size], workspace[size:]
    y = rsm.ssm_prefill(x, dt, A, B, C, i32(cu), st, initial_slots=i32([0] + [-1] * (S - 1)),
                        final_slots=i32(list(range(1, S + 1))), D=D, device_status=status, workspace=workspace)
    assert int(status) == rsm.STATUS_BITS["bad_sequence"]
    assert bool((beyond == 77).all())
    wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, [0, T], before, [0], D)
    base.close(y, wy, base.HALF_UNIT[inputs], wm, base.y_terms(inputs, T), "y")
    base.close(st[1:2], ws, base.HALF_UNIT[F32], wsm, base.state_terms(inputs, F32, T), "state")
    assert torch.equal(st[0], before[0]) and torch.equal(st[2:], before[2:])
    if case != "cut":  # (cut for another number of sequences, sums differ in their order)
        assert torch.equal(y, want) and torch.equal(st[1], first[1])


@pytest.mark.parametrize("case", ["cut", "longest first", "one by one"])
def test_prefill_runs_what_is_good_before_bad_sequences(case):
    """Sequences that start before the tokens, that end past them, and a step back, around good ones."""
    H, G = 2, 1
    n, inputs = {"cut": (2000, BF16), "longest first": (150, BF16), "one by one": (40, F32)}[case]
    T = 3 * n
    cu = [-9, -5, 0, n, n, 2 * n, T + 1, T + 7, 2 * n, T]
    good = {2: (0, n), 3: (n, n), 4: (n, 2 * n)}
    S = len(cu) - 1
    x, dt, A, B, C, D = base.tokens((T,), H, G, 64, 128, inputs, 5)
    st = base.pool(2 * S, H, 64, 128, F32, 6)
    before, status = st.clone(), word()
    out = torch.full_like(x, 9.0)
    rsm.ssm_prefill(x, dt, A, B, C, i32(cu), st, initial_slots=i32(list(range(S))), final_slots=i32(list(range(S, 2 * S))),
                    D=D, device_status=status, out=out)
    assert int(status) == rsm.STATUS_BITS["bad_sequence"]
    for s, (a, b) in good.items():
        if a == b:
            assert torch.equal(st[S + s], before[s])
            continue
        wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, [a, b], before, [s], D)
        base.close(out[a:b], wy[a:b], base.HALF_UNIT[inputs], wm[a:b], base.y_terms(inputs, n), "y")
        base.close(st[S + s:S + s + 1], ws, base.HALF_UNIT[F32], wsm, base.state_terms(inputs, F32, n), "state")
    keep = [i for i in range(2 * S) if i - S not in good]
    assert torch.equal(st[keep], before[keep]) and bool((out[2 * n:] == 9).all())


def test_decode_from_two_threads():
    """Rings of 50 and of 64 rows run on one kernel with different amounts of shared memory; neither thread's calls
    are refused for the other's, and each gets what it gets alone."""
    H, T = 2, 4
    lib, calls = block._load(), []
    for R in (50, 64):
        x, dt, A, B, C, D = base.tokens((1, T), H, 1, 64, 128, F32, R)
        xc, dtc, _, Bc, _, _ = base.tokens((1, R), H, 1, 64, 128, F32, R + 1)
        st, zero, have = base.pool(1, H, 64, 128, BF16, R + 2), i32([0]), i32([5])
        want = rsm.replayssm_decode(st, zero, xc, Bc, dtc, zero, have, x, dt, A, B, C, D=D)
        out = torch.zeros_like(x)
        a = block.ReplaySsmDecodeArgs()
        tensors = dict(x=x, B=B, C=C, dt=dt, A=A, D=D, state=st, x_cache=xc, B_cache=Bc, dt_cache=dtc, slots=zero,
                       ring_start=zero, ring_len=have, out=out)
        for name, t in tensors.items():
            setattr(a, name, t.data_ptr())
        for name, t in (("x", x), ("B", B), ("C", C), ("dt", dt)):
            setattr(a, name + "_batch_stride", t.stride(0))
            setattr(a, name + "_stride", t.stride(1))
        for name, t in (("state", st), ("x_cache", xc), ("B_cache", Bc), ("dt_cache", dtc)):
            setattr(a, name + "_slot_stride", t.stride(0))
        a.batch, a.window, a.num_slots, a.num_heads, a.num_groups, a.dim, a.dstate, a.ring_buffer_len = 1, T, 1, H, 1, 64, 128, R
        a.state_dtype, a.input_dtype, a.pad_slot_id = rsm.RSM_BF16, rsm.RSM_F32, -1
        calls.append((bytes(a), want, tensors))
    torch.cuda.synchronize()
    stream, refused, together = torch.cuda.current_stream().cuda_stream, [], threading.Barrier(2)

    def work(args):
        torch.cuda.set_device(0)
        together.wait()
        for k in range(20000):
            rc = lib.rsm_replayssm_decode(args, stream)
            if rc != 0:
                refused.append((rc, lib.rsm_block_last_error().decode()))
            if k % 200 == 199:
                torch.cuda.synchronize()

    threads = [threading.Thread(target=work, args=(c[0],)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, f"{len(refused)} calls refused: {refused[0]}"
    assert all(torch.equal(c[2]["out"], c[1]) for c in calls)


def test_prefill_flags_a_bad_initial_slot_of_a_cut_sequence():
    """One long sequence of few heads, cut into segments: a slot out of range starts from zero and is flagged, the
    pad starts from zero and is not."""
    T, H = 3001, 2
    assert prefill_workspace(T, 1, H, 1) > 0
    x, dt, A, B, C, D = base.tokens((T,), H, 1, 64, 128, BF16, 3)
    st = base.pool(3, H, 64, 128, F32, 4)
    out = []
    for slot, bits in ((-1, 0), (3, rsm.STATUS_BITS["bad_slot"]), (-7, rsm.STATUS_BITS["bad_slot"])):
        status, pool = word(), st.clone()
        out.append((rsm.ssm_prefill(x, dt, A, B, C, i32([0, T]), pool, initial_slots=i32([slot]), final_slots=i32([2]),
                                    D=D, device_status=status), pool))
        assert int(status) == bits, slot
    assert all(torch.equal(y, out[0][0]) and torch.equal(p, out[0][1]) for y, p in out)


def check_decays(rates, state=F32, size=1.0, T=300, skip=True):
    """A prompt whose tokens decay by rates [T, H] nats, with x, B and C of about `size`."""
    H = rates.shape[1]
    x, _, _, B, C, D = base.tokens((T,), H, 1, 64, 128, BF16, 8)
    x, B, C = x * size, B * size, C * size
    A = -(0.5 + torch.rand(H, generator=base.gen(9), device="cuda"))
    dt = (rates / -A).float()
    st = base.pool(2, H, 64, 128, state, 10)
    before = st.clone()
    D = D if skip else None
    y = rsm.ssm_prefill(x, dt, A, B, C, i32([0, T]), st, initial_slots=i32([0]), final_slots=i32([1]), D=D)
    wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, [0, T], before, [0], D)
    base.close(y, wy, 2.0 ** -8, wm, base.y_terms(BF16, T), "y")
    base.close(st[1:], ws, base.HALF_UNIT[state], wsm, base.state_terms(BF16, state, T), "state")


LN2 = 0.6931471805599453


@pytest.mark.parametrize("log2", [20.0, 31.0, 33.0, 40.0, 90.0, 99.5, 100.5, 140.0])
@pytest.mark.parametrize("size", [1.0, 4096.0, 2.0 ** -20])
def test_prefill_decays_of_a_half_chunk(log2, size):
    """64 tokens decay by about 2^-log2, on either side of where the kernel changes its way, values small and large
    (sums from 2^-60 to 2^45 are far inside every type here)."""
    g = base.gen(11)
    rates = LN2 * log2 / 64 * (0.8 + 0.4 * torch.rand((300, 4), generator=g, device="cuda"))
    check_decays(rates, size=size)
    check_decays(torch.full((300, 3), LN2 * log2 / 64, device="cuda"), state=BF16, size=size, skip=False)


@pytest.mark.parametrize("heads", [[0], [1], [1, 2]])
@pytest.mark.parametrize("halves", [[0], [1], [2, 3], [0, 3], [1, 2]])
def test_prefill_steep_heads_and_halves_mixed(heads, halves):
    """Some heads, and some halves of their chunks, decay by more than 2^-100, their neighbours mildly."""
    g = base.gen(12)
    rates = 0.001 + 0.1 * torch.rand((300, 4), generator=g, device="cuda")
    for h in heads:
        for k in halves:
            rates[64 * k:64 * k + 64, h] = 1.2 + torch.rand(64, generator=g, device="cuda")
    check_decays(rates)
    check_decays(rates, state=BF16, size=64.0)


def test_prefill_one_steep_token():
    """A single token that decays everything before it to nothing, first, in the middle or last of a half."""
    for at in (0, 31, 32, 63, 64, 100, 127, 128, 255):
        rates = 0.001 + 0.1 * torch.rand((300, 3), generator=base.gen(13), device="cuda")
        rates[at, 1] = 150.0
        check_decays(rates)


@pytest.mark.parametrize("state", [F32, F16, BF16])
@pytest.mark.parametrize("inf", [float("inf"), -float("inf")])
def test_an_infinite_input_leaves_an_infinite_state(state, inf):
    """S += dt x (x) B with one infinite x: that row of the state is infinite with B's signs, and nothing else is."""
    H, d, h = 4, 5, 3
    for way in ("prompt", "step"):
        T, at = (40, 10) if way == "prompt" else (4, 1)
        x, dt, A, B, C, D = base.tokens((T,), H, 2, 64, 128, BF16, 5)
        B = torch.where(B == 0, torch.ones_like(B), B)
        x[at, h, d] = inf
        st = base.pool(2, H, 64, 128, state, 6)
        before = st.clone()
        if way == "prompt":
            y = rsm.ssm_prefill(x, dt, A, B, C, i32([0, T]), st, initial_slots=i32([0]), final_slots=i32([1]), D=D)
        else:
            y = rsm.ssm_step(st, i32([0]), x[None], dt[None], A, B[None], C[None], dst_slots=i32([1]), D=D)[0]
        wy, wm, ws, wsm = ref.prefill(x, dt, A, B, C, [0, T], before, [0], D)
        assert torch.equal(st[1, h, d].double(), ws[0, h, d]) and bool(torch.isinf(ws[0, h, d]).all()), way
        keep = torch.ones(H, 64, dtype=torch.bool, device="cuda")
        keep[h, d] = False
        base.close(st[1][keep], ws[0][keep], base.HALF_UNIT[state], wsm[0][keep], base.state_terms(BF16, state, T), "state")
        base.close(y[:, keep], wy[:, keep], 2.0 ** -8, wm[:, keep], base.y_terms(BF16, T), "y")


@pytest.mark.parametrize("state", [F32, F16, BF16])
@pytest.mark.parametrize("T", [1, 2, 12])
def test_an_infinite_state_is_read_as_one(state, T):
    """One infinite element of a checkpoint: its row's outputs are infinite with C's signs, the others as ever."""
    H, d, h, n = 4, 9, 2, 77
    x, dt, A, B, C, D = base.tokens((1, T), H, 2, 64, 128, BF16, 5)
    C = torch.where(C == 0, torch.ones_like(C), C)
    xc, dtc, _, Bc, _, _ = base.tokens((1, 16), H, 2, 64, 128, BF16, 6)
    st = base.pool(1, H, 64, 128, state, 7)
    args = lambda s: (s, i32([0]), xc.clone(), Bc.clone(), dtc.clone(), i32([2]), i32([3]), x, dt, A, B, C)  # noqa: E731
    clean = rsm.replayssm_decode(*args(st), D=D)
    st2 = st.clone()
    st2[0, h, d, n] = float("inf")
    y = rsm.replayssm_decode(*args(st2), D=D)
    assert torch.equal(y[0, :, h, d].double(), C[0, :, h // 2, n].double() * float("inf"))
    y[0, :, h, d] = clean[0, :, h, d]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("inputs", [F32, BF16])
@pytest.mark.parametrize("early", ["ring", "new"])
def test_decode_mild_tokens_after_strong_ones(inputs, early):
    """Tokens whose decay is mild, after ring rows or new tokens that decay the state to nothing: a pair's decay is
    what lies between its tokens, whatever lies before."""
    R, T, H, G = 64, 8, 4, 2
    have = R - T if early == "ring" else 1
    x, dt, A, B, C, D = base.tokens((1, T), H, G, 64, 128, inputs, 1)
    xc, dtc, _, Bc, _, _ = base.tokens((1, R), H, G, 64, 128, inputs, 2)
    A = -(16.0 + 16.0 * torch.rand(H, generator=base.gen(3), device="cuda"))
    dtc, dt = 0.1 * dtc, 0.1 * dt
    strong = 4.0 + 4.0 * torch.rand((40, H), generator=base.gen(4), device="cuda")
    if early == "ring":
        dtc[0, :40] = strong
    else:
        dt[0, :4] = strong[:4] * 40.0
    st = base.pool(1, H, 64, 128, F32, 5)
    y = rsm.replayssm_decode(st, i32([0]), xc.clone(), Bc.clone(), dtc.clone(), i32([0]), i32([have]), x, dt, A, B, C, D=D)
    cat = lambda c, t: torch.cat([ref.f64(c[0, :have]), ref.f64(t[0])])  # noqa: E731
    S = ref.f64(st[0])
    Cs = torch.cat([torch.zeros(have, G, 128, dtype=torch.float64, device="cuda"), ref.f64(C[0])])
    wy, wm, _, _ = ref.run_tokens(S, S.abs(), cat(xc, x), cat(dtc, dt), ref.f64(A), cat(Bc, B), Cs, ref.f64(D))
    base.close(y[0], wy[have:], base.HALF_UNIT[inputs], wm[have:], base.y_terms(inputs, R), "y")


def every_call(T=2):
    """The operators with a pad slot, as functions of it."""
    x, dt, A, B, C, D = base.tokens((3, T), 4, 2, 64, 128, BF16, 1)
    xc, dtc, _, Bc, _, _ = base.tokens((3, 8), 4, 2, 64, 128, BF16, 2)
    st = base.pool(3, 4, 64, 128, F32, 3)
    slots, zero = i32([0, 1, 2]), i32([0, 0, 0])
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    return {
        "prefill": lambda **k: rsm.ssm_prefill(flat(x), flat(dt), A, flat(B), flat(C), i32([0, 1, 2, 3 * T]), st,
                                               initial_slots=slots, final_slots=slots, **k),
        "step": lambda **k: rsm.ssm_step(st, slots, x, dt, A, B, C, **k),
        "decode": lambda **k: rsm.replayssm_decode(st, slots, xc, Bc, dtc, zero, zero, x, dt, A, B, C, **k)}


@pytest.mark.parametrize("name", ["prefill", "step", "decode"])
@pytest.mark.parametrize("pad", [2 ** 32 - 1, 2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_a_pad_slot_past_32_bits_is_refused(name, pad):
    call = every_call()[name]
    with pytest.raises(ValueError, match="pad_slot_id"):
        call(pad_slot_id=pad)


def test_a_group_size_past_32_bits_is_refused():
    x, w = torch.ones(2, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="group_size"):
        rsm.gated_rms_norm(x, x, w, group_size=2 ** 32 + 64)


def grad_calls():
    """(operator, its tensor arguments that could want a gradient)."""
    x, dt, A, B, C, D = base.tokens((3, 2), 4, 2, 64, 128, BF16, 1)
    xc, dtc, _, Bc, _, _ = base.tokens((3, 8), 4, 2, 64, 128, BF16, 2)
    st = base.pool(3, 4, 64, 128, F32, 3)
    slots, zero = i32([0, 1, 2]), i32([0, 0, 0])
    flat = lambda t: t.detach().flatten(0, 1).requires_grad_(t.requires_grad)  # noqa: E731
    g, r, w = torch.randn(4, 64, device="cuda"), torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    return [
        (lambda x, dt, A, B, C, D, **k: rsm.ssm_prefill(flat(x), flat(dt), A, flat(B), flat(C), i32([0, 6]), D=D, **k),
         [x, dt, A, B, C, D]),
        (lambda x, dt, A, B, C, D, **k: rsm.ssm_step(st.clone(), slots, x, dt, A, B, C, D=D, **k), [x, dt, A, B, C, D]),
        (lambda x, dt, A, B, C, D, **k: rsm.replayssm_decode(st, slots, xc.clone(), Bc.clone(), dtc.clone(), zero, zero, x,
                                                             dt, A, B, C, D=D, **k), [x, dt, A, B, C, D]),
        (lambda x, r, w, **k: rsm.add_rms_norm(x, r, w, **k)[0], [g, r, w]),
        (lambda x, z, w, **k: rsm.gated_rms_norm(x, z, w, **k), [g, r, w])]


@pytest.mark.parametrize("op", range(5), ids=["prefill", "step", "decode", "add_norm", "gated_norm"])
def test_a_gradient_that_would_be_lost_is_refused(op):
    """The operators are forward only: an input that wants a gradient is refused while gradients are recorded, by
    either way into the library, and served as ever where they are not."""
    call, tensors = grad_calls()[op]
    want = call(*tensors)
    for i, t in enumerate(tensors):
        args = [*tensors[:i], t.clone().requires_grad_(), *tensors[i + 1:]]
        for way in ({}, {"out": torch.empty_like(want)}):
            with pytest.raises(ValueError, match="forward only"):
                call(*args, **way)
            with torch.no_grad():
                assert torch.equal(call(*args, **way), want)


def test_a_skipped_request_of_a_window_past_32_bit_offsets_is_zero():
    """Its output rows hold more than 2^31 values (4.3 GB)."""
    T = (1 << 31) // 16 + 3
    x = torch.zeros((1, 1, 1, 16), dtype=BF16, device="cuda").expand(1, T, 1, 16)
    dt = torch.zeros((1, 1, 1), device="cuda").expand(1, T, 1)
    out = torch.full((1, T, 1, 16), 7.0, dtype=BF16, device="cuda")
    st = torch.zeros((1, 1, 16, 16), device="cuda")
    rsm.ssm_step(st, i32([-1]), x, dt, torch.zeros(1, device="cuda"), x, x, out=out)
    assert not bool(out.any())


def same_both_ways(make, call):
    """The call with and without a status word (marshalled by block.py, and by _blockcall): equal to the bit."""
    a, b = make(), make()
    ya, yb = call(a, device_status=word()), call(b)
    assert torch.equal(ya, yb)
    for p, q in zip(a, b):
        assert p is q or p is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("state", [F32, BF16, F16, torch.int8, torch.float8_e4m3fn], ids=str)
@pytest.mark.parametrize("inputs,T,sliced,skip", [(BF16, 1, 0, True), (BF16, 4, 3, False), (F32, 2, 8, True), (BF16, 0, 0, False)])
def test_decode_marshalled_either_way(state, inputs, T, sliced, skip):
    """T = 0: tokens without the window dimension."""
    b, R, H, G = 4, 16, 6, 2
    x, dt, A, B, C, D = base.tokens((b, T) if T else (b,), H, G, 64, 128, inputs, 3, sliced)
    xc, dtc, _, Bc, _, _ = base.tokens((b + 1, R), H, G, 64, 128, inputs, 4)
    scale = None
    if state in (torch.int8, torch.float8_e4m3fn):
        st = torch.randint(-127, 128, (b + 1, H, 64, 128), generator=base.gen(5), device="cuda", dtype=torch.int8)
        st = st if state == torch.int8 else st.to(F16).to(state)
        scale = 0.01 + 0.05 * torch.rand((b + 1, H, 64), generator=base.gen(6), device="cuda")
    else:
        st = base.pool(b + 1, H, 64, 128, state, 5)
    same_both_ways(lambda: (st.clone(), xc.clone(), Bc.clone(), dtc.clone()),
                   lambda m, **k: rsm.replayssm_decode(m[0], i32([3, -1, 1, 4]), *m[1:], i32([0, 3, 15, 9]), i32([5, 0, 12, 1]),
                                                       x, dt, A, B, C, state_scale=scale, D=D if skip else None, **k))


@pytest.mark.parametrize("state", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("inputs,T,sliced,skip", [(BF16, 1, 0, True), (BF16, 4, 3, False), (F32, 2, 8, True), (BF16, 0, 0, False)])
@pytest.mark.parametrize("in_place", [True, False])
def test_step_marshalled_either_way(state, inputs, T, sliced, skip, in_place):
    b, H, G = 4, 6, 2
    x, dt, A, B, C, D = base.tokens((b, T) if T else (b,), H, G, 64, 128, inputs, 3, sliced)
    st = base.pool(2 * b, H, 64, 128, state, 5)
    same_both_ways(lambda: (st.clone(),),
                   lambda m, **k: rsm.ssm_step(m[0], i32([3, -1, 1, 0]), x, dt, A, B, C, dst_slots=None if in_place else i32([7, 6, -1, 4]),
                                               D=D if skip else None, **k))


@pytest.mark.parametrize("state", [F32, BF16, F16, None], ids=str)
@pytest.mark.parametrize("inputs,lens,sliced,skip", [(BF16, [3], 0, True), (BF16, [140, 0, 33], 8, False), (F32, [20, 7], 0, True),
                                                     (BF16, [30, 90], 3, True), (BF16, [2500], 0, False)])
def test_prefill_marshalled_either_way(state, inputs, lens, sliced, skip):
    S, H, G = len(lens), 6, 2
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0, dtype=torch.int32)
    x, dt, A, B, C, D = base.tokens((sum(lens),), H, G, 64, 128, inputs, 3, sliced)
    st = None if state is None else base.pool(2 * S, H, 64, 128, state, 5)
    final = list(range(2 * S - 1, S - 1, -1))
    if S > 1:
        final[-1] = -1
    slots = {} if state is None else dict(initial_slots=i32([-1] + list(range(1, S))), final_slots=i32(final))
    same_both_ways(lambda: (None if st is None else st.clone(),),
                   lambda m, **k: rsm.ssm_prefill(x, dt, A, B, C, cu, m[0], D=D if skip else None, **slots, **k))


def test_calls_recorded_in_a_graph():
    """Each operator as a graph replays it, results and workspaces from the graph's pool, on inputs that changed since."""
    x, dt, A, B, C, D = base.tokens((2500,), 4, 2, 64, 128, BF16, 1)
    xt, dtt, _, Bt, Ct, _ = base.tokens((2, 3), 4, 2, 64, 128, BF16, 2)
    xc, dtc, _, Bc, _, _ = base.tokens((2, 16), 4, 2, 64, 128, BF16, 3)
    st, w = base.pool(2, 4, 64, 128, F32, 4), torch.ones(256, device="cuda")
    cu, slots, start, have = i32([0, 2500]), i32([0, 1]), i32([3, 9]), i32([2, 5])
    rows = torch.randn(4, 256, device="cuda")
    results = lambda: (rsm.ssm_prefill(x, dt, A, B, C, cu, D=D), rsm.ssm_step(st, slots, xt, dtt, A, Bt, Ct, D=D),  # noqa: E731
                       rsm.replayssm_decode(st, slots, xc, Bc, dtc, start, have, xt, dtt, A, Bt, Ct, D=D),
                       *rsm.add_rms_norm(rows, rows, w), rsm.gated_rms_norm(rows, rows, w))
    before = st.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        results()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        recorded = results()
    for t in (x, xt, rows):
        t.neg_()
    st.copy_(before)
    graph.replay()
    got = [t.clone() for t in recorded]
    st.copy_(before)
    for a, b in zip(got, results()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("inputs", [BF16, F32])
def test_rows_that_no_token_reaches_may_hold_anything(inputs):
    """NaN in ring rows outside the window, in other slots, in tokens of no sequence and in a skipped request."""
    nan = float("nan")
    x, dt, A, B, C, D = base.tokens((3, 2), 4, 2, 64, 128, inputs, 1)
    xc, dtc, _, Bc, _, _ = base.tokens((4, 16), 4, 2, 64, 128, inputs, 2)
    st = base.pool(4, 4, 64, 128, F32, 3)
    args = lambda s, x, B, C, dt, c: (s, i32([2, -1, 0]), *c, i32([14, 0, 3]), i32([5, 0, 0]), x, dt, A, B, C)  # noqa: E731
    clean = [t.clone() for t in (xc, Bc, dtc)]
    want = rsm.replayssm_decode(*args(st, x, B, C, dt, clean), D=D)
    used = torch.zeros(4, 16, dtype=torch.bool, device="cuda")
    used[2, [14, 15, 0, 1, 2]] = True
    dirty = [torch.where(used.view(4, 16, *[1] * (t.dim() - 2)), t, nan) for t in (xc, Bc, dtc)]
    st2, x2, B2, C2, dt2 = (t.clone() for t in (st, x, B, C, dt))
    st2[[1, 3]] = nan
    for t in (x2, B2, C2, dt2):
        t[1] = nan
    assert torch.equal(rsm.replayssm_decode(*args(st2, x2, B2, C2, dt2, dirty), D=D), want)
    for n in (5, 40, 150):
        p = base.tokens((200,), 4, 2, 64, 128, inputs, 4)
        want = rsm.ssm_prefill(*p[:5], i32([20, 20 + n]), D=p[5])[20:20 + n].clone()
        for t in (p[0], p[1], p[3], p[4]):
            t[:20] = nan
            t[20 + n:] = nan
        assert torch.equal(rsm.ssm_prefill(*p[:5], i32([20, 20 + n]), D=p[5])[20:20 + n], want)
