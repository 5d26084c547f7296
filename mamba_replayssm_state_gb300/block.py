"""The operators of the layer around replayssm_materialize, forward only.

Linear attention with a decay for each head, in its three serving forms:
  ssm_prefill        packed prompts, chunked
  ssm_step           new tokens of running requests, state slot to state slot
  replayssm_decode   new tokens from a checkpoint slot and its replay ring; the
                     state is only read, the ring is written, and
                     replayssm_materialize commits the accepted prefix later
and the norms around the layer: add_rms_norm before it, gated_rms_norm after it.

Each call checks its tensors, passes their addresses and strides to the C ABI
(include/replayssm_block.h, which states the semantics) and enqueues the
kernels on the current CUDA stream, or on `stream`.  Results and workspaces
that the caller does not pass are allocated on that stream.  There is no
fallback: without the library the calls raise.  While gradients are recorded,
a tensor that requires one is refused: there is no backward pass to take it.

The usual calls (the current stream, results allocated, no status word, tensors
as the kernels take them) are checked and marshalled by _blockcall, a C++
extension: 11 to 21 us a call on the GB300's Arm host are then 4 to 6.  What it
does not take comes back to the code here, which names what is wrong or lets it
pass, through ctypes.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import RSM_F32, ReplaySSMError, _dtype_code, load_library

__all__ = ["ssm_prefill", "ssm_step", "replayssm_decode", "add_rms_norm", "gated_rms_norm"]

_CTYPE = {"P": ctypes.c_void_p, "q": ctypes.c_int64, "i": ctypes.c_int32, "f": ctypes.c_float}


def _mirror(name, *fields):
    """A ctypes mirror of a C struct and the packer of its bytes, from (type code, field names) pairs."""
    flat = [(f, c) for c, names in fields for f in names.split()]
    cls = type(name, (ctypes.Structure,), {"_fields_": [(f, _CTYPE[c]) for f, c in flat]})
    fmt = struct.Struct("@" + "".join(c for _, c in flat) + "0q")
    return cls, fmt.pack, fmt.size


SsmPrefillArgs, _pack_prefill, _n0 = _mirror(
    "SsmPrefillArgs", ("P", "x B C dt A D cu_seqlens state initial_slots final_slots out workspace device_status"),
    ("q", "tokens x_stride B_stride C_stride dt_stride out_stride state_slot_stride workspace_bytes"),
    ("i", "num_seqs num_slots num_heads num_groups dim dstate state_dtype input_dtype pad_slot_id"))
SsmStepArgs, _pack_step, _n1 = _mirror(
    "SsmStepArgs", ("P", "x B C dt A D state src_slots dst_slots out device_status"),
    ("q", "x_batch_stride x_stride B_batch_stride B_stride C_batch_stride C_stride dt_batch_stride dt_stride "
          "state_slot_stride"),
    ("i", "batch window num_slots num_heads num_groups dim dstate state_dtype input_dtype pad_slot_id"))
ReplaySsmDecodeArgs, _pack_decode, _n2 = _mirror(
    "ReplaySsmDecodeArgs",
    ("P", "x B C dt A D state state_scale x_cache B_cache dt_cache slots ring_start ring_len out device_status"),
    ("q", "x_batch_stride x_stride B_batch_stride B_stride C_batch_stride C_stride dt_batch_stride dt_stride "
          "state_slot_stride scale_slot_stride x_cache_slot_stride B_cache_slot_stride dt_cache_slot_stride"),
    ("i", "batch window num_slots num_heads num_groups dim dstate ring_buffer_len state_dtype input_dtype pad_slot_id"))
AddRmsNormArgs, _pack_add, _n3 = _mirror(
    "AddRmsNormArgs", ("P", "x residual weight out residual_out"),
    ("q", "rows x_stride residual_stride out_stride residual_out_stride"), ("i", "dim input_dtype residual_dtype"),
    ("f", "residual_scale eps"))
GatedRmsNormArgs, _pack_gated, _n4 = _mirror(
    "GatedRmsNormArgs", ("P", "x z weight out"), ("q", "rows x_stride z_stride out_stride"),
    ("i", "dim group_size input_dtype norm_before_gate"), ("f", "eps"), ("i", "reserved"))

_calls = None

ARGS = (SsmPrefillArgs, SsmStepArgs, ReplaySsmDecodeArgs, AddRmsNormArgs, GatedRmsNormArgs)
_lib = None


def _load():
    global _lib, _calls
    if _lib is None:
        lib = load_library()
        _calls = _load_calls()
        for i, (cls, n) in enumerate(zip(ARGS, (_n0, _n1, _n2, _n3, _n4))):
            if not lib.rsm_block_args_size(i) == ctypes.sizeof(cls) == n:
                raise OSError(f"{cls.__name__} layout mismatch between libreplayssm.so and the binding")
        for f in ("rsm_ssm_prefill", "rsm_ssm_step", "rsm_replayssm_decode", "rsm_add_rms_norm", "rsm_gated_rms_norm"):
            getattr(lib, f).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            getattr(lib, f).restype = ctypes.c_int
        lib.rsm_ssm_prefill_workspace.argtypes = [ctypes.c_char_p]
        lib.rsm_ssm_prefill_workspace.restype = ctypes.c_int64
        lib.rsm_block_last_error.restype = ctypes.c_char_p
        _calls.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
            "rsm_ssm_prefill", "rsm_ssm_prefill_workspace", "rsm_ssm_step", "rsm_replayssm_decode", "rsm_add_rms_norm",
            "rsm_gated_rms_norm")))
        _lib = lib
    return _lib


def _load_calls():
    """_blockcall, built first where it is missing or older than its source."""
    from . import _build
    _build.build_calls()
    from . import _blockcall
    return _blockcall


def _raise(name, rc):
    e = ReplaySSMError(rc, "")
    e.args = (f"{name} failed ({rc}): {_lib.rsm_block_last_error().decode()}",)
    raise e


_INPUTS = {torch.bfloat16: _dtype_code(torch.bfloat16), torch.float32: RSM_F32}
_STATES = {t: _dtype_code(t) for t in (torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn)}
_I32, _F32 = torch.int32, torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice

# A decode step makes a few of these calls a layer, so what a call checks it
# checks first in one expression that the usual tensors pass; only where that
# fails do the _check functions go over it, and name what is wrong or let it pass
# (strides of dimensions of one element, for instance).


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _check_device(*tensors):
    """All tensors are on the current CUDA device."""
    devices = {t.get_device() for t in tensors if t is not None}
    _need(devices != set() and min(devices) >= 0, "tensors must be CUDA tensors")
    _need(len(devices) == 1, "all tensors must be on one CUDA device")
    _need(devices == {torch.cuda.current_device()}, "tensors must be on the current CUDA device")


def _check_grad(*tensors):
    """None wants a gradient that the call would not pass on."""
    if torch.is_grad_enabled():
        _need(not any(t is not None and t.requires_grad for t in tensors),
              "the operators are forward only, and a tensor requires a gradient: detach it, or call under torch.no_grad()")


def _check_rows(t, name, shape, inner, dtype):
    """t has the shape, and its last `inner` dimensions are contiguous."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    size = 1
    for n, stride in zip(reversed(shape[len(shape) - inner:]), reversed(t.stride())):
        if n != 1 and stride != size:
            raise ValueError(f"{name} must be contiguous in its last {inner} dimension(s)")
        size *= n


def _check_vector(t, name, n, dtype):
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values")


def _check_tokens(x, dt, A, B, C, D, k):
    """The token tensors, with k leading dimensions."""
    _need(x.dtype in _INPUTS, f"x must be bfloat16 or float32, got {x.dtype}")
    _need(x.dim() == k + 2 and B.dim() == k + 2, f"x and B must have {k + 2} dimensions")
    lead, heads, groups = x.shape[:k], x.shape[k:], B.shape[k:]
    _check_rows(x, "x", (*lead, *heads), 2, x.dtype)
    _check_rows(B, "B", (*lead, *groups), 2, x.dtype)
    _check_rows(C, "C", (*lead, *groups), 2, x.dtype)
    _check_rows(dt, "dt", (*lead, heads[0]), 1, _F32)
    _check_vector(A, "A", heads[0], _F32)
    if D is not None:
        _check_vector(D, "D", heads[0], _F32)


def _check_state(state, H, dim, N):
    _need(state.dtype in _STATES, f"unsupported state dtype {state.dtype}")
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, dim, N) or not state[0:1].is_contiguous():
        raise ValueError(f"state must be [slots, {H}, {dim}, {N}] with contiguous slots, got {list(state.shape)}")


def _check_out(out, x):
    if out.dtype != x.dtype or out.shape != x.shape:
        raise ValueError(f"out must be {x.dtype} {list(x.shape)}")


def _int32(value, name):
    value = int(value)
    _need(-2 ** 31 <= value < 2 ** 31, f"{name} must fit 32 bits, got {value}")
    return value


def _status(t):
    if t is None:
        return 0
    _need(t.numel() == 1 and t.element_size() == 4, "device_status must be one 32-bit word")
    return t.data_ptr()


def _handle(stream, device):
    """The raw handle of `stream`, or of the current one."""
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new_on(stream, make):
    """A tensor of the stream that the kernels run on."""
    if hasattr(stream, "cuda_stream"):
        with torch.cuda.stream(stream):
            return make()
    if int(stream) != _raw_stream(_current_device()):
        raise ValueError("a raw stream handle needs the results to be passed in (out=...)")
    return make()


def _like(x, stream):
    """A contiguous tensor like x."""
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _new_on(stream, lambda: torch.empty_like(x, memory_format=torch.contiguous_format))


def ssm_prefill(x, dt, A, B, C, cu_seqlens, state=None, *, initial_slots=None, final_slots=None, D=None,
                pad_slot_id=-1, out=None, workspace=None, device_status=None, stream=None):
    """Linear attention with a decay for each head over packed prompts.

    x [tokens, H, dim], B and C [tokens, G, dstate] (bf16 or fp32), dt
    [tokens, H], A [H], D [H] or None (fp32); cu_seqlens [seqs + 1] int32.
    Sequence s starts from state[initial_slots[s]] (default: from zero) and
    leaves its state in state[final_slots[s]] (default: nowhere), a slot that is
    no other sequence's; the pool `state` is [slots, H, dim, dstate] fp32, bf16 or
    fp16.  Returns the outputs, [tokens, H, dim].  A long call of few sequences needs a workspace, which is
    allocated where `workspace` (a contiguous uint8 CUDA tensor) is not given.
    """
    lib = _lib or _load()
    if stream is None and out is None and workspace is None and device_status is None:
        r = _calls.prefill(x, dt, A, B, C, cu_seqlens, state, initial_slots, final_slots, D, pad_slot_id)
        if r is not None:
            return r if type(r) is not int else _raise("ssm_prefill", r)
    _check_grad(x, dt, A, B, C, D, state, out)
    sx, sB, sC, sd = x.stride(), B.stride(), C.stride(), dt.stride()
    shape, code, dev = x.shape, _INPUTS.get(x.dtype), x.get_device()
    if not (code is not None and len(shape) == 3 and B.shape == C.shape and len(sB) == 3 and dt.shape == shape[:2]
            and shape[0] == B.shape[0] and x.dtype is B.dtype and x.dtype is C.dtype and dt.dtype is _F32
            and A.dtype is _F32 and A.shape == shape[1:2] and A.is_contiguous() and sx[2] == 1 and sx[1] == shape[2]
            and sB[2] == 1 and sB[1] == B.shape[2] and sC[2] == 1 and sC[1] == B.shape[2] and sd[1] == 1
            and (D is None or (D.dtype is _F32 and D.shape == shape[1:2] and D.is_contiguous()))):
        _check_tokens(x, dt, A, B, C, D, 1)
    T, H, dim = shape
    G, N = B.shape[1:]
    seqs = cu_seqlens.shape[0] - 1
    _need(seqs >= 0, "cu_seqlens must have at least one entry")
    if not (dev >= 0 and dev == B.get_device() == C.get_device() == dt.get_device() == A.get_device()
            == cu_seqlens.get_device() and dev == _current_device()
            and D is None and state is None and device_status is None and workspace is None and out is None):
        _check_device(x, dt, A, B, C, D, cu_seqlens, state, initial_slots, final_slots, out, workspace, device_status)
    _check_vector(cu_seqlens, "cu_seqlens", seqs + 1, _I32)
    sd_code, ss, slots, ps, pi, pf = RSM_F32, 0, 0, 0, 0, 0
    if state is not None:
        _check_state(state, H, dim, N)
        sd_code, ss, slots, ps = _STATES[state.dtype], state.stride(0), state.shape[0], state.data_ptr()
    else:
        _need(initial_slots is None and final_slots is None, "slots need a state pool")
    if initial_slots is not None:
        _check_vector(initial_slots, "initial_slots", seqs, _I32)
        pi = initial_slots.data_ptr()
    if final_slots is not None:
        _check_vector(final_slots, "final_slots", seqs, _I32)
        pf = final_slots.data_ptr()
    if out is None:
        out, so = _like(x, stream), H * dim
    else:
        _check_out(out, x)
        _check_rows(out, "out", shape, 2, x.dtype)
        so = out.stride(0)
        _need(T < 2 or so >= H * dim, "rows of out overlap")
    args = [x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), A.data_ptr(), 0 if D is None else D.data_ptr(),
            cu_seqlens.data_ptr(), ps, pi, pf, out.data_ptr(), 0, _status(device_status), T, sx[0], sB[0], sC[0], sd[0],
            so, ss, 0, seqs, slots, H, G, dim, N, sd_code, code, _int32(pad_slot_id, "pad_slot_id")]
    packed = _pack_prefill(*args)
    size = lib.rsm_ssm_prefill_workspace(packed)
    if size < 0:
        _raise("ssm_prefill", size)
    if size > 0:
        if workspace is None:
            make = lambda: torch.empty(size, dtype=torch.uint8, device=x.device)  # noqa: E731
            workspace = make() if stream is None else _new_on(stream, make)
        _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(), "workspace must be a contiguous uint8 tensor")
        args[11], args[20] = workspace.data_ptr(), workspace.numel()
        packed = _pack_prefill(*args)
    rc = lib.rsm_ssm_prefill(packed, _handle(stream, dev))
    if rc != 0:
        _raise("ssm_prefill", rc)
    return out


def _batch(x, dt, A, B, C, D):
    """Checks the token tensors of running requests, with or without the window dimension; the input code, (batch,
    window, H, G, dim, dstate) and the batch and token strides of x, B, C and dt."""
    sx, sB, sC, sd = x.stride(), B.stride(), C.stride(), dt.stride()
    shape, bshape, code, k = x.shape, B.shape, _INPUTS.get(x.dtype), len(sx) - 2
    _need(k in (1, 2), "x must be [batch, window, H, dim] or [batch, H, dim]")
    if not (code is not None and len(sB) == k + 2 and bshape == C.shape and bshape[:k] == shape[:k]
            and dt.shape == shape[:-1] and x.dtype is B.dtype and x.dtype is C.dtype and dt.dtype is _F32
            and A.dtype is _F32 and A.shape == shape[k:-1] and A.is_contiguous() and sx[-1] == 1 and sx[-2] == shape[-1]
            and sB[-1] == 1 and sB[-2] == bshape[-1] and sC[-1] == 1 and sC[-2] == bshape[-1] and sd[-1] == 1
            and (D is None or (D.dtype is _F32 and D.shape == A.shape and D.is_contiguous()))):
        _check_tokens(x, dt, A, B, C, D, k)
    if k == 1:
        return (code, shape[0], 1, shape[1], bshape[1], shape[2], bshape[2], sx[0], 0, sB[0], 0, sC[0], 0, sd[0], 0)
    return (code, shape[0], shape[1], shape[2], bshape[2], shape[3], bshape[3], sx[0], sx[1], sB[0], sB[1], sC[0], sC[1],
            sd[0], sd[1])


def ssm_step(state, slots, x, dt, A, B, C, *, dst_slots=None, D=None, pad_slot_id=-1, out=None, device_status=None,
             stream=None):
    """The new tokens of running requests, in the recurrent form.

    x [batch, window, H, dim], dt [batch, window, H], B and C [batch, window, G,
    dstate]; without the window dimension, one token each.  The tokens are
    applied in order to state[slots[b]] and the result is stored to
    state[dst_slots[b]] (default: in place); destinations are distinct and no
    other request's source.  Returns the outputs, shaped like x; rows of a
    request with the pad slot are zero.
    """
    lib = _lib or _load()
    if stream is None and out is None and device_status is None:
        r = _calls.step(state, slots, x, dt, A, B, C, dst_slots, D, pad_slot_id)
        if r is not None:
            return r if type(r) is not int else _raise("ssm_step", r)
    _check_grad(x, dt, A, B, C, D, state, out)
    code, b, T, H, G, dim, N, *strides = _batch(x, dt, A, B, C, D)
    dev = x.get_device()
    if not (dev >= 0 and dev == B.get_device() == C.get_device() == dt.get_device() == A.get_device()
            == state.get_device() == slots.get_device() and dev == _current_device() and device_status is None
            and (D is None or D.get_device() == dev) and (dst_slots is None or dst_slots.get_device() == dev)
            and (out is None or out.get_device() == dev)):
        _check_device(x, dt, A, B, C, D, state, slots, dst_slots, out, device_status)
    sd = _STATES.get(state.dtype)
    if not (sd is not None and state.is_contiguous() and state.shape[1:] == (H, dim, N)):
        _check_state(state, H, dim, N)
    if not (slots.dtype is _I32 and slots.shape == (b,) and slots.is_contiguous()):
        _check_vector(slots, "slots", b, _I32)
    pd = 0
    if dst_slots is not None:
        if not (dst_slots.dtype is _I32 and dst_slots.shape == (b,) and dst_slots.is_contiguous()):
            _check_vector(dst_slots, "dst_slots", b, _I32)
        pd = dst_slots.data_ptr()
    if out is None:
        out = _like(x, stream)
    else:
        _check_out(out, x)
        _need(out.is_contiguous(), "out must be contiguous")
    rc = lib.rsm_ssm_step(_pack_step(
        x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), A.data_ptr(), 0 if D is None else D.data_ptr(),
        state.data_ptr(), slots.data_ptr(), pd, out.data_ptr(), _status(device_status), *strides, state.stride(0), b, T,
        state.shape[0], H, G, dim, N, sd, code, _int32(pad_slot_id, "pad_slot_id")), _handle(stream, dev))
    if rc != 0:
        _raise("ssm_step", rc)
    return out


def _check_cache(t, name, shape, dtype):
    if t.dtype != dtype or tuple(t.shape) != shape or not t[0:1].is_contiguous():
        raise ValueError(f"{name} must be {dtype} {list(shape)} with contiguous slots")


def replayssm_decode(state, slots, x_cache, B_cache, dt_cache, ring_start, ring_len, x, dt, A, B, C, *,
                     state_scale=None, D=None, pad_slot_id=-1, out=None, device_status=None, stream=None):
    """New tokens from a checkpoint state and its replay ring; the state is only read.

    Request b's state is state[slots[b]] advanced by ring rows ring_start[b] ..
    ring_start[b] + ring_len[b] - 1 (modulo the ring's length); the new tokens
    (x, dt, B, C as for ssm_step) follow, and are written to the ring rows after
    those.  The slots are distinct.  The caller advances ring_len.  Caches are one layer's x [slots, R, H,
    dim], B [slots, R, G, dstate] and dt [slots, R, H], as replayssm_materialize
    reads them; one-byte states come with state_scale [slots, H, dim].
    Returns the outputs, shaped like x; rows of a skipped request are zero.
    """
    lib = _lib or _load()
    if stream is None and out is None and device_status is None:
        r = _calls.decode(state, slots, x_cache, B_cache, dt_cache, ring_start, ring_len, x, dt, A, B, C, state_scale, D,
                          pad_slot_id)
        if r is not None:
            return r if type(r) is not int else _raise("replayssm_decode", r)
    _check_grad(x, dt, A, B, C, D, state, x_cache, B_cache, dt_cache, state_scale, out)
    code, b, T, H, G, dim, N, *strides = _batch(x, dt, A, B, C, D)
    dev = x.get_device()
    if not (dev >= 0 and dev == B.get_device() == C.get_device() == dt.get_device() == A.get_device()
            == state.get_device() == slots.get_device() == x_cache.get_device() == B_cache.get_device()
            == dt_cache.get_device() == ring_start.get_device() == ring_len.get_device() and dev == _current_device()
            and device_status is None and (D is None or D.get_device() == dev)
            and (state_scale is None or state_scale.get_device() == dev) and (out is None or out.get_device() == dev)):
        _check_device(x, dt, A, B, C, D, state, slots, x_cache, B_cache, dt_cache, ring_start, ring_len, state_scale,
                      out, device_status)
    sd, sshape, xshape = _STATES.get(state.dtype), state.shape, x_cache.shape
    if not (sd is not None and state.is_contiguous() and sshape[1:] == (H, dim, N)):
        _check_state(state, H, dim, N)
    S = sshape[0]
    _need(len(xshape) == 4, "x_cache must be [slots, R, H, dim]")
    R = xshape[1]
    if not (x_cache.dtype is x.dtype and xshape == (S, R, H, dim) and x_cache.is_contiguous()
            and B_cache.dtype is x.dtype and B_cache.shape == (S, R, G, N) and B_cache.is_contiguous()
            and dt_cache.dtype is _F32 and dt_cache.shape == (S, R, H) and dt_cache.is_contiguous()):
        _check_cache(x_cache, "x_cache", (S, R, H, dim), x.dtype)
        _check_cache(B_cache, "B_cache", (S, R, G, N), x.dtype)
        _check_cache(dt_cache, "dt_cache", (S, R, H), _F32)
    if not (slots.dtype is _I32 and slots.shape == (b,) and slots.is_contiguous()
            and ring_start.dtype is _I32 and ring_start.shape == (b,) and ring_start.is_contiguous()
            and ring_len.dtype is _I32 and ring_len.shape == (b,) and ring_len.is_contiguous()):
        for name, t in (("slots", slots), ("ring_start", ring_start), ("ring_len", ring_len)):
            _check_vector(t, name, b, _I32)
    pq, sq = 0, 0
    if state_scale is not None:
        _check_cache(state_scale, "state_scale", (S, H, dim), _F32)
        pq, sq = state_scale.data_ptr(), state_scale.stride(0)
    if out is None:
        out = _like(x, stream)
    else:
        _check_out(out, x)
        _need(out.is_contiguous(), "out must be contiguous")
    rc = lib.rsm_replayssm_decode(_pack_decode(
        x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), A.data_ptr(), 0 if D is None else D.data_ptr(),
        state.data_ptr(), pq, x_cache.data_ptr(), B_cache.data_ptr(), dt_cache.data_ptr(), slots.data_ptr(),
        ring_start.data_ptr(), ring_len.data_ptr(), out.data_ptr(), _status(device_status), *strides, state.stride(0), sq,
        x_cache.stride(0), B_cache.stride(0), dt_cache.stride(0), b, T, S, H, G, dim, N, R, sd, code,
        _int32(pad_slot_id, "pad_slot_id")), _handle(stream, dev))
    if rc != 0:
        _raise("replayssm_decode", rc)
    return out


def _rows(t, name, shape, dtype):
    """(address, row stride) of a [..., dim] tensor seen as rows."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    if len(shape) == 2:
        if shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
        return t.data_ptr(), t.stride(0)
    try:
        v = t.view(-1, shape[-1])
    except RuntimeError:
        raise ValueError(f"the leading dimensions of {name} must be one stride apart") from None
    return _rows(v, name, v.shape, dtype)


def _result(out, name, like, shape, stream):
    """(tensor, address, row stride) of a result like `like`."""
    if out is None:
        out = _like(like, stream)
        return out, out.data_ptr(), shape[-1]
    ptr, stride = _rows(out, name, shape, like.dtype)
    _need(out.numel() <= shape[-1] or stride >= shape[-1], f"rows of {name} overlap")
    return out, ptr, stride


def add_rms_norm(x, residual, weight, *, residual_scale=1.0, eps=1e-5, out=None, residual_out=None, stream=None):
    """The norm before a block: r = residual + residual_scale * x; returns
    (r / sqrt(mean(r^2) + eps) * weight, r) over the last dimension.

    x is bf16 or fp32 (and so is the norm), residual bf16 or fp32 (and so is
    r), weight fp32.  `out` may be x, `residual_out` may be residual.
    """
    lib = _lib or _load()
    if stream is None and out is None and residual_out is None:
        r = _calls.add_norm(x, residual, weight, residual_scale, eps)
        if r is not None:
            return r if type(r) is not int else _raise("add_rms_norm", r)
    _check_grad(x, residual, weight, out, residual_out)
    shape, code, rcode, dev = x.shape, _INPUTS.get(x.dtype), _INPUTS.get(residual.dtype), x.get_device()
    _need(len(shape) >= 1 and shape[-1] > 0, "x must have a last dimension")
    _need(code is not None and rcode is not None, "x and residual must be bfloat16 or float32")
    if not (dev >= 0 and dev == residual.get_device() == weight.get_device() and dev == _current_device()
            and out is None and residual_out is None):
        _check_device(x, residual, weight, out, residual_out)
    dim = shape[-1]
    px, sx = _rows(x, "x", shape, x.dtype)
    pr, sr = _rows(residual, "residual", shape, residual.dtype)
    _check_vector(weight, "weight", dim, _F32)
    out, po, so = _result(out, "out", x, shape, stream)
    residual_out, pq, sq = _result(residual_out, "residual_out", residual, shape, stream)
    rc = lib.rsm_add_rms_norm(_pack_add(px, pr, weight.data_ptr(), po, pq, x.numel() // dim, sx, sr, so, sq, dim, code,
                                        rcode, float(residual_scale), float(eps)), _handle(stream, dev))
    if rc != 0:
        _raise("add_rms_norm", rc)
    return out, residual_out


def gated_rms_norm(x, z, weight, *, group_size=None, eps=1e-5, norm_before_gate=False, out=None, stream=None):
    """The norm after a block, over groups of `group_size` of the last
    dimension (default: all of it): x silu(z) normalised and weighted, or, with
    norm_before_gate, x normalised and weighted, then times silu(z).

    x and z are bf16 or fp32, alike, weight fp32.  `out` may be x.
    """
    lib = _lib or _load()
    if stream is None and out is None:
        r = _calls.gated_norm(x, z, weight, group_size, eps, norm_before_gate)
        if r is not None:
            return r if type(r) is not int else _raise("gated_rms_norm", r)
    _check_grad(x, z, weight, out)
    shape, code, dev = x.shape, _INPUTS.get(x.dtype), x.get_device()
    _need(len(shape) >= 1 and shape[-1] > 0, "x must have a last dimension")
    _need(code is not None, f"x must be bfloat16 or float32, got {x.dtype}")
    if not (dev >= 0 and dev == z.get_device() == weight.get_device() and dev == _current_device() and out is None):
        _check_device(x, z, weight, out)
    dim = shape[-1]
    px, sx = _rows(x, "x", shape, x.dtype)
    pz, sz = _rows(z, "z", shape, x.dtype)
    _check_vector(weight, "weight", dim, _F32)
    out, po, so = _result(out, "out", x, shape, stream)
    rc = lib.rsm_gated_rms_norm(_pack_gated(px, pz, weight.data_ptr(), po, x.numel() // dim, sx, sz, so, dim,
                                            dim if group_size is None else _int32(group_size, "group_size"), code,
                                            1 if norm_before_gate else 0, float(eps), 0), _handle(stream, dev))
    if rc != 0:
        _raise("gated_rms_norm", rc)
    return out
