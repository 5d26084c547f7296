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
fallback: without the library the calls raise.
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

ARGS = (SsmPrefillArgs, SsmStepArgs, ReplaySsmDecodeArgs, AddRmsNormArgs, GatedRmsNormArgs)
_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = load_library()
        for i, (cls, n) in enumerate(zip(ARGS, (_n0, _n1, _n2, _n3, _n4))):
            if not lib.rsm_block_args_size(i) == ctypes.sizeof(cls) == n:
                raise OSError(f"{cls.__name__} layout mismatch between libreplayssm.so and the binding")
        for f in ("rsm_ssm_prefill", "rsm_ssm_step", "rsm_replayssm_decode", "rsm_add_rms_norm", "rsm_gated_rms_norm"):
            getattr(lib, f).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            getattr(lib, f).restype = ctypes.c_int
        lib.rsm_ssm_prefill_workspace.argtypes = [ctypes.c_char_p]
        lib.rsm_ssm_prefill_workspace.restype = ctypes.c_int64
        lib.rsm_block_last_error.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def _raise(name, rc):
    e = ReplaySSMError(rc, "")
    e.args = (f"{name} failed ({rc}): {_lib.rsm_block_last_error().decode()}",)
    raise e


_INPUTS = {torch.bfloat16: _dtype_code(torch.bfloat16), torch.float32: RSM_F32}
_STATES = {t: _dtype_code(t) for t in (torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn)}
_I32, _F32 = torch.int32, torch.float32


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _device(x, *others):
    """The CUDA device index all the tensors are on, which has to be the current one."""
    d = x.get_device()
    _need(d >= 0, "tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors must be on one CUDA device")
    _need(d == torch.cuda.current_device(), "tensors must be on the current CUDA device")
    return d


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream):
    """A result tensor of the stream that the kernels run on."""
    if stream is not None and hasattr(stream, "cuda_stream"):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    if stream is not None and int(stream) != torch._C._cuda_getCurrentRawStream(device.index):
        raise ValueError("a raw stream handle needs the results to be passed in (out=...)")
    return torch.empty(shape, dtype=dtype, device=device)


def _input(t, name, lead, inner, dtype):
    """Checks a [*lead, *inner] tensor whose inner dimensions are contiguous."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != (*lead, *inner):
        raise ValueError(f"{name} must be {[*lead, *inner]}, got {list(t.shape)}")
    s = t.stride()
    if (s[-1] != 1 and inner[-1] != 1) or (len(inner) == 2 and s[-2] != inner[1] and inner[0] != 1):
        raise ValueError(f"{name} must be contiguous in its last {len(inner)} dimension(s)")
    return s


def _vector(t, name, n, dtype):
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values")
    return t.data_ptr()


def _status(t):
    if t is None:
        return None
    _need(t.numel() == 1 and t.element_size() == 4, "device_status must be one 32-bit word")
    return t.data_ptr()


def _heads(x, dt, A, B, C, D, lead):
    """Checks the token tensors; (heads, groups, dim, dstate, input code, their strides, A, D)."""
    k = len(lead)
    _need(x.dim() == k + 2 and B.dim() == k + 2, f"x and B must have {k + 2} dimensions")
    code = _INPUTS.get(x.dtype)
    _need(code is not None, f"x must be bfloat16 or float32, got {x.dtype}")
    H, dim = x.shape[k:]
    G, N = B.shape[k:]
    sx, sB = _input(x, "x", lead, (H, dim), x.dtype), _input(B, "B", lead, (G, N), x.dtype)
    sC, sdt = _input(C, "C", lead, (G, N), x.dtype), _input(dt, "dt", lead, (H,), _F32)
    a = _vector(A, "A", H, _F32)
    d = None if D is None else _vector(D, "D", H, _F32)
    return H, G, dim, N, code, sx, sB, sC, sdt, a, d


def _state(state, H, dim, N):
    code = _STATES.get(state.dtype)
    _need(code is not None, f"unsupported state dtype {state.dtype}")
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, dim, N) or not state[0:1].is_contiguous():
        raise ValueError(f"state must be [slots, {H}, {dim}, {N}] with contiguous slots, got {list(state.shape)}")
    return code


def _out(out, x, shape, stream):
    if out is None:
        return _empty(shape, x.dtype, x.device, stream)
    if out.dtype != x.dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {x.dtype} {list(shape)}")
    return out


def ssm_prefill(x, dt, A, B, C, cu_seqlens, state=None, *, initial_slots=None, final_slots=None, D=None,
                pad_slot_id=-1, out=None, workspace=None, device_status=None, stream=None):
    """Linear attention with a decay for each head over packed prompts.

    x [tokens, H, dim], B and C [tokens, G, dstate] (bf16 or fp32), dt
    [tokens, H], A [H], D [H] or None (fp32); cu_seqlens [seqs + 1] int32.
    Sequence s starts from state[initial_slots[s]] (default: from zero) and
    leaves its state in state[final_slots[s]] (default: nowhere); the pool
    `state` is [slots, H, dim, dstate] fp32, bf16 or fp16.  Returns the outputs,
    [tokens, H, dim].  `workspace` (optional) is a uint8 CUDA tensor of at least
    ssm_prefill_workspace_bytes(...) bytes.
    """
    lib = _lib or _load()
    T = x.shape[0]
    H, G, dim, N, code, sx, sB, sC, sdt, a, d = _heads(x, dt, A, B, C, D, (T,))
    dev = _device(x, dt, A, B, C, D, cu_seqlens, state, initial_slots, final_slots, out, workspace, device_status)
    seqs = cu_seqlens.shape[0] - 1
    _need(seqs >= 0, "cu_seqlens must have at least one entry")
    _need(state is not None or (initial_slots is None and final_slots is None), "slots need a state pool")
    sd, ss, slots = (RSM_F32, 0, 0) if state is None else (_state(state, H, dim, N), state.stride(0), state.shape[0])
    out = _out(out, x, (T, H, dim), stream)
    so = _input(out, "out", (T,), (H, dim), x.dtype)
    _need(T < 2 or so[0] >= H * dim, "rows of out overlap")
    args = [x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), a, d or 0,
            _vector(cu_seqlens, "cu_seqlens", seqs + 1, _I32), 0 if state is None else state.data_ptr(),
            0 if initial_slots is None else _vector(initial_slots, "initial_slots", seqs, _I32),
            0 if final_slots is None else _vector(final_slots, "final_slots", seqs, _I32), out.data_ptr(), 0,
            _status(device_status) or 0, T, sx[0], sB[0], sC[0], sdt[0], so[0], ss, 0, seqs, slots, H, G, dim, N, sd,
            code, int(pad_slot_id)]
    size = lib.rsm_ssm_prefill_workspace(_pack_prefill(*args))
    if size < 0:
        _raise("ssm_prefill", size)
    if size > 0:
        if workspace is None:
            workspace = _empty((size,), torch.uint8, x.device, stream)
        _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(), "workspace must be a contiguous uint8 tensor")
        args[11], args[20] = workspace.data_ptr(), workspace.numel()
    rc = lib.rsm_ssm_prefill(_pack_prefill(*args), _stream(stream, dev))
    if rc != 0:
        _raise("ssm_prefill", rc)
    return out


def ssm_step(state, slots, x, dt, A, B, C, *, dst_slots=None, D=None, pad_slot_id=-1, out=None, device_status=None,
             stream=None):
    """The new tokens of running requests, in the recurrent form.

    x [batch, window, H, dim], dt [batch, window, H], B and C [batch, window, G,
    dstate]; without the window dimension, one token each.  The tokens are
    applied in order to state[slots[b]] and the result is stored to
    state[dst_slots[b]] (default: in place).  Returns the outputs, shaped like
    x; rows of a request with the pad slot are zero.
    """
    lib = _lib or _load()
    one = x.dim() == 3
    if one:
        x, dt, B, C = x.unsqueeze(1), dt.unsqueeze(1), B.unsqueeze(1), C.unsqueeze(1)
        out = None if out is None else out.unsqueeze(1)
    b, T = x.shape[:2]
    H, G, dim, N, code, sx, sB, sC, sdt, a, d = _heads(x, dt, A, B, C, D, (b, T))
    dev = _device(x, dt, A, B, C, D, state, slots, dst_slots, out, device_status)
    sd = _state(state, H, dim, N)
    out = _out(out, x, (b, T, H, dim), stream)
    _need(out.is_contiguous(), "out must be contiguous")
    rc = lib.rsm_ssm_step(_pack_step(
        x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), a, d or 0, state.data_ptr(),
        _vector(slots, "slots", b, _I32), 0 if dst_slots is None else _vector(dst_slots, "dst_slots", b, _I32),
        out.data_ptr(), _status(device_status) or 0, sx[0], sx[1], sB[0], sB[1], sC[0], sC[1], sdt[0], sdt[1],
        state.stride(0), b, T, state.shape[0], H, G, dim, N, sd, code, int(pad_slot_id)), _stream(stream, dev))
    if rc != 0:
        _raise("ssm_step", rc)
    return out.squeeze(1) if one else out


def replayssm_decode(state, slots, x_cache, B_cache, dt_cache, ring_start, ring_len, x, dt, A, B, C, *,
                     state_scale=None, D=None, pad_slot_id=-1, out=None, device_status=None, stream=None):
    """New tokens from a checkpoint state and its replay ring; the state is only read.

    Request b's state is state[slots[b]] advanced by ring rows ring_start[b] ..
    ring_start[b] + ring_len[b] - 1 (modulo the ring's length); the new tokens
    (x, dt, B, C as for ssm_step) follow, and are written to the ring rows after
    those.  The caller advances ring_len.  Caches are one layer's x [slots, R, H,
    dim], B [slots, R, G, dstate] and dt [slots, R, H], as replayssm_materialize
    reads them; one-byte states come with state_scale [slots, H, dim].
    Returns the outputs, shaped like x; rows of a skipped request are zero.
    """
    lib = _lib or _load()
    one = x.dim() == 3
    if one:
        x, dt, B, C = x.unsqueeze(1), dt.unsqueeze(1), B.unsqueeze(1), C.unsqueeze(1)
        out = None if out is None else out.unsqueeze(1)
    b, T = x.shape[:2]
    H, G, dim, N, code, sx, sB, sC, sdt, a, d = _heads(x, dt, A, B, C, D, (b, T))
    dev = _device(x, dt, A, B, C, D, state, slots, x_cache, B_cache, dt_cache, ring_start, ring_len, state_scale, out,
                  device_status)
    sd = _state(state, H, dim, N)
    S = state.shape[0]
    _need(x_cache.dim() == 4, "x_cache must be [slots, R, H, dim]")
    R = x_cache.shape[1]
    for name, t, shape, dtype in (("x_cache", x_cache, (S, R, H, dim), x.dtype), ("B_cache", B_cache, (S, R, G, N), x.dtype),
                                  ("dt_cache", dt_cache, (S, R, H), _F32)):
        if t.dtype != dtype or tuple(t.shape) != shape or not t[0:1].is_contiguous():
            raise ValueError(f"{name} must be {dtype} {list(shape)} with contiguous slots")
    if state_scale is not None and (state_scale.dtype != _F32 or tuple(state_scale.shape) != (S, H, dim)
                                    or not state_scale[0:1].is_contiguous()):
        raise ValueError(f"state_scale must be float32 {[S, H, dim]} with contiguous slots")
    out = _out(out, x, (b, T, H, dim), stream)
    _need(out.is_contiguous(), "out must be contiguous")
    rc = lib.rsm_replayssm_decode(_pack_decode(
        x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), a, d or 0, state.data_ptr(),
        0 if state_scale is None else state_scale.data_ptr(), x_cache.data_ptr(), B_cache.data_ptr(),
        dt_cache.data_ptr(), _vector(slots, "slots", b, _I32), _vector(ring_start, "ring_start", b, _I32),
        _vector(ring_len, "ring_len", b, _I32), out.data_ptr(), _status(device_status) or 0, sx[0], sx[1], sB[0],
        sB[1], sC[0], sC[1], sdt[0], sdt[1], state.stride(0), 0 if state_scale is None else state_scale.stride(0),
        x_cache.stride(0), B_cache.stride(0), dt_cache.stride(0), b, T, S, H, G, dim, N, R, sd, code,
        int(pad_slot_id)), _stream(stream, dev))
    if rc != 0:
        _raise("replayssm_decode", rc)
    return out.squeeze(1) if one else out


def _rows(t, name, shape, dtype):
    """(address, row stride) of a [..., dim] tensor seen as rows."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.dim() == 2:
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
        return t.data_ptr(), t.stride(0)
    try:
        v = t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"the leading dimensions of {name} must be one stride apart") from None
    return _rows(v, name, v.shape, dtype)


def add_rms_norm(x, residual, weight, *, residual_scale=1.0, eps=1e-5, out=None, residual_out=None, stream=None):
    """The norm before a block: r = residual + residual_scale * x; returns
    (r / sqrt(mean(r^2) + eps) * weight, r) over the last dimension.

    x is bf16 or fp32 (and so is the norm), residual bf16 or fp32 (and so is
    r), weight fp32.  `out` may be x, `residual_out` may be residual.
    """
    lib = _lib or _load()
    _need(x.dim() >= 1 and x.shape[-1] > 0, "x must have a last dimension")
    code, rcode = _INPUTS.get(x.dtype), _INPUTS.get(residual.dtype)
    _need(code is not None and rcode is not None, "x and residual must be bfloat16 or float32")
    dev = _device(x, residual, weight, out, residual_out)
    dim, shape = x.shape[-1], x.shape
    out = _out(out, x, shape, stream)
    residual_out = _out(residual_out, residual, shape, stream)
    (px, sx), (pr, sr) = _rows(x, "x", shape, x.dtype), _rows(residual, "residual", shape, residual.dtype)
    (po, so), (pq, sq) = _rows(out, "out", shape, x.dtype), _rows(residual_out, "residual_out", shape, residual.dtype)
    _need(x.numel() <= dim or (so >= dim and sq >= dim), "rows of out or residual_out overlap")
    rc = lib.rsm_add_rms_norm(_pack_add(px, pr, _vector(weight, "weight", dim, _F32), po, pq, x.numel() // dim, sx, sr,
                                        so, sq, dim, code, rcode, float(residual_scale), float(eps)),
                              _stream(stream, dev))
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
    _need(x.dim() >= 1 and x.shape[-1] > 0, "x must have a last dimension")
    code = _INPUTS.get(x.dtype)
    _need(code is not None, f"x must be bfloat16 or float32, got {x.dtype}")
    dev = _device(x, z, weight, out)
    dim, shape = x.shape[-1], x.shape
    out = _out(out, x, shape, stream)
    (px, sx), (pz, sz), (po, so) = (_rows(x, "x", shape, x.dtype), _rows(z, "z", shape, x.dtype),
                                    _rows(out, "out", shape, x.dtype))
    _need(x.numel() <= dim or so >= dim, "rows of out overlap")
    rc = lib.rsm_gated_rms_norm(_pack_gated(px, pz, _vector(weight, "weight", dim, _F32), po, x.numel() // dim, sx, sz,
                                            so, dim, dim if group_size is None else int(group_size), code,
                                            int(bool(norm_before_gate)), float(eps), 0), _stream(stream, dev))
    if rc != 0:
        _raise("gated_rms_norm", rc)
    return out
