"""The operators of a hybrid stack around the layer operators of block.py, forward only.

  causal_conv        the short convolution before the state space operator, packed prompts
  causal_conv_step   the same for new tokens of running requests, drafts among them
  rotary_append      rotary positions on q and k of new tokens; k and v go to their pages
  paged_attention    new tokens over their requests' pages of keys and values
  copy_pages         pages of all layers' pools copied in one call
  rotary_frequencies the inverse frequencies that rotary_append takes, also for longer contexts

Rows of the caches go by a token's position in its request: a draft that is rejected
costs nothing to undo, the next call starts at an earlier position and writes over it.

Calls check, allocate and fail as block.py's do, with the C ABI of
include/replayssm_hybrid.h, which states the semantics; their usual forms are checked and
marshalled by _hybridcall, a C++ extension.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _dtype_code, load_library
from .block import (_F32, _I32, _INPUTS, _STATES, _check_device, _check_grad, _check_out, _check_rows, _check_vector, _handle,
                    _int32, _like, _mirror, _need, _new_on, _status, ReplaySSMError)

__all__ = ["causal_conv", "causal_conv_step", "rotary_append", "paged_attention", "copy_pages", "rotary_frequencies"]

CausalConvArgs, _pack_conv, _n0 = _mirror(
    "CausalConvArgs", ("P", "x weight bias cu_seqlens cache slots positions out device_status"),
    ("q", "tokens x_stride out_stride cache_slot_stride"),
    ("i", "num_seqs num_slots channels width cache_rows input_dtype silu pad_slot_id"))
CausalConvStepArgs, _pack_conv_step, _n1 = _mirror(
    "CausalConvStepArgs", ("P", "x weight bias cache slots positions out device_status"),
    ("q", "x_batch_stride x_stride cache_slot_stride"),
    ("i", "batch window num_slots channels width cache_rows input_dtype silu pad_slot_id reserved"))
_PAGES = (("P", "k_pages v_pages page_table lengths"),
          ("q", "k_page_stride k_row_stride k_head_stride v_page_stride v_row_stride v_head_stride table_stride"),
          ("i", "requests table_width num_pages page_size"))
RotaryAppendArgs, _pack_rotary, _n2 = _mirror(
    "RotaryAppendArgs", ("P", "q k v inv_freq cu_seqlens q_out device_status"), *_PAGES,
    ("q", "tokens q_batch_stride q_stride k_batch_stride k_stride v_batch_stride v_stride out_batch_stride out_stride"),
    ("i", "window num_heads num_kv_heads dim rotary_dim input_dtype interleaved"), ("f", "amplitude"))
PagedAttentionArgs, _pack_attention, _n3 = _mirror(
    "PagedAttentionArgs", ("P", "q out workspace device_status"), *_PAGES,
    ("q", "q_batch_stride q_stride workspace_bytes"), ("i", "window num_heads num_kv_heads dim input_dtype"), ("f", "scale"))
CopyPagesArgs, _pack_copy, _n4 = _mirror(
    "CopyPagesArgs", ("P", "page_ptrs page_strides src_pages dst_pages device_status"), ("q", "page_elements"),
    ("i", "num_pools num_pairs num_pages dtype"))

ARGS = (CausalConvArgs, CausalConvStepArgs, RotaryAppendArgs, PagedAttentionArgs, CopyPagesArgs)
_lib = None
_calls = None


def _load():
    global _lib, _calls
    if _lib is None:
        lib = load_library()
        from . import _build
        _build.build_calls()
        from . import _hybridcall
        for i, (cls, n) in enumerate(zip(ARGS, (_n0, _n1, _n2, _n3, _n4))):
            if not lib.rsm_hybrid_args_size(i) == ctypes.sizeof(cls) == n:
                raise OSError(f"{cls.__name__} layout mismatch between libreplayssm.so and the binding")
        names = ("rsm_causal_conv", "rsm_causal_conv_step", "rsm_rotary_append", "rsm_paged_attention",
                 "rsm_paged_attention_workspace", "rsm_copy_pages")
        for f in names:
            getattr(lib, f).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            getattr(lib, f).restype = ctypes.c_int
        lib.rsm_paged_attention_workspace.argtypes = [ctypes.c_char_p]
        lib.rsm_paged_attention_workspace.restype = ctypes.c_int64
        lib.rsm_hybrid_last_error.restype = ctypes.c_char_p
        _hybridcall.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in names))
        _calls, _lib = _hybridcall, lib
    return _lib


def _raise(name, rc):
    e = ReplaySSMError(rc, "")
    e.args = (f"{name} failed ({rc}): {_lib.rsm_hybrid_last_error().decode()}",)
    raise e


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _check_taps(x, weight, bias):
    _need(x.dtype in _INPUTS, f"x must be bfloat16 or float32, got {x.dtype}")
    C = x.shape[-1]
    _need(C > 0, "x must have channels")
    _need(C == 1 or x.stride(-1) == 1, "x must be contiguous in its last dimension")
    _need(weight.dtype == _F32 and weight.dim() == 2 and weight.shape[0] == C and weight.is_contiguous(),
          f"weight must be a contiguous float32 tensor [{C}, width]")
    if bias is not None:
        _check_vector(bias, "bias", C, _F32)


def _check_conv_cache(cache, x):
    _need(cache.dtype == x.dtype and cache.dim() == 3 and cache.shape[2] == x.shape[-1] and cache[0:1].is_contiguous(),
          f"cache must be {x.dtype} [slots, rows, {x.shape[-1]}] with contiguous slots")
    _need(cache.shape[0] < 2 or cache.stride(0) >= cache.shape[1] * cache.shape[2], "slots of the cache overlap")


def causal_conv(x, weight, cu_seqlens, bias=None, cache=None, slots=None, positions=None, *, silu=True, pad_slot_id=-1,
                out=None, device_status=None, stream=None):
    """The short causal convolution over packed prompts, each channel on its own, and silu.

    x [tokens, channels] (bf16 or fp32; x, B and C of a layer are one slice of its
    projection), weight [channels, width] (2, 3 or 4) and bias [channels] fp32,
    cu_seqlens [seqs + 1] int32.  cache [slots, rows, channels], of x's type, keeps the
    inputs by position, row position mod rows (rows >= width - 1): sequence s's tokens are at
    positions positions[s] (default 0) and up, its earlier inputs in slot slots[s],
    where its last width - 1 are left.  Returns the outputs, [tokens, channels].
    """
    lib = _lib or _load()
    if stream is None and out is None and device_status is None:
        r = _calls.conv(x, weight, cu_seqlens, bias, cache, slots, positions, silu, pad_slot_id)
        if r is not None:
            return r if type(r) is not int else _raise("causal_conv", r)
    _check_grad(x, weight, bias, cache, out)
    _need(x.dim() == 2, "x must be [tokens, channels]")
    _check_taps(x, weight, bias)
    _check_device(x, weight, bias, cu_seqlens, cache, slots, positions, out, device_status)
    seqs = cu_seqlens.shape[0] - 1
    _need(seqs >= 0, "cu_seqlens must have at least one entry")
    _check_vector(cu_seqlens, "cu_seqlens", seqs + 1, _I32)
    _need((cache is None) == (slots is None), "cache and slots go together")
    _need(cache is not None or positions is None, "positions need a cache")
    ss = n = rows = 0
    if cache is not None:
        _check_conv_cache(cache, x)
        _check_vector(slots, "slots", seqs, _I32)
        if positions is not None:
            _check_vector(positions, "positions", seqs, _I32)
        ss, (n, rows) = cache.stride(0), cache.shape[:2]
    T, C = x.shape
    if out is None:
        out, so = _like(x, stream), C
    else:
        _check_out(out, x)
        _check_rows(out, "out", x.shape, 1, x.dtype)
        so = out.stride(0)
        _need(T < 2 or so >= C, "rows of out overlap")
    rc = lib.rsm_causal_conv(_pack_conv(
        x.data_ptr(), weight.data_ptr(), _ptr(bias), cu_seqlens.data_ptr(), _ptr(cache), _ptr(slots), _ptr(positions),
        out.data_ptr(), _status(device_status), T, x.stride(0), so, ss, seqs, n, C, weight.shape[1], rows, _INPUTS[x.dtype],
        bool(silu), _int32(pad_slot_id, "pad_slot_id")), _handle(stream, x.get_device()))
    if rc != 0:
        _raise("causal_conv", rc)
    return out


def causal_conv_step(x, weight, cache, slots, positions, bias=None, *, silu=True, pad_slot_id=-1, out=None,
                     device_status=None, stream=None):
    """causal_conv for the new tokens of running requests.

    x [batch, window, channels], or [batch, channels] for one token each; request b's
    tokens are at positions positions[b] and up, its earlier inputs in slot slots[b] of
    the cache, where all the new ones are stored (rows >= width - 1 + window).  If only some
    of them are accepted, the next call's position says so.  Slots are distinct; rows of a
    request with the pad slot are zero.  Returns the outputs, shaped like x.
    """
    lib = _lib or _load()
    if stream is None and out is None and device_status is None:
        r = _calls.conv_step(x, weight, cache, slots, positions, bias, silu, pad_slot_id)
        if r is not None:
            return r if type(r) is not int else _raise("causal_conv_step", r)
    _check_grad(x, weight, bias, cache, out)
    _need(x.dim() in (2, 3), "x must be [batch, window, channels] or [batch, channels]")
    _check_taps(x, weight, bias)
    _check_device(x, weight, bias, cache, slots, positions, out, device_status)
    _check_conv_cache(cache, x)
    b, C, T = x.shape[0], x.shape[-1], x.shape[1] if x.dim() == 3 else 1
    _check_vector(slots, "slots", b, _I32)
    _check_vector(positions, "positions", b, _I32)
    if out is None:
        out = _like(x, stream)
    else:
        _check_out(out, x)
        _need(out.is_contiguous(), "out must be contiguous")
    rc = lib.rsm_causal_conv_step(_pack_conv_step(
        x.data_ptr(), weight.data_ptr(), _ptr(bias), cache.data_ptr(), slots.data_ptr(), positions.data_ptr(),
        out.data_ptr(), _status(device_status), x.stride(0), x.stride(1) if x.dim() == 3 else 0, cache.stride(0), b, T,
        cache.shape[0], C, weight.shape[1], cache.shape[1], _INPUTS[x.dtype], bool(silu),
        _int32(pad_slot_id, "pad_slot_id"), 0), _handle(stream, x.get_device()))
    if rc != 0:
        _raise("causal_conv_step", rc)
    return out


def _check_heads(t, name, dtype, lead, heads, dim):
    _check_rows(t, name, (*lead, heads, dim), 2, dtype)


def _pages(k_cache, v_cache, page_table, lengths, dtype, dim, requests):
    """Checks a layer's pages; their part of an argument struct, in _PAGES' order."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t.dtype == dtype and t.dim() == 4 and t.shape[3] == dim and t.shape == k_cache.shape,
              f"{name} must be {dtype} [pages, page_size, kv_heads, {dim}], and k_cache and v_cache of one shape")
        _need(dim == 1 or t.stride(3) == 1, f"{name} must be contiguous in its last dimension")
        need = dim
        for stride, n in sorted((s, n) for n, s in zip(t.shape[:3], t.stride()) if n > 1):
            _need(stride >= need, f"rows of {name} overlap")
            need = stride * n
    _need(page_table.dtype == _I32 and page_table.dim() == 2 and page_table.shape[0] == requests
          and (page_table.shape[1] < 2 or page_table.stride(1) == 1),
          f"page_table must be an int32 tensor [{requests}, pages of a request] with contiguous rows")
    _check_vector(lengths, "lengths", requests, _I32)
    return ((k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr()),
            (*k_cache.stride()[:3], *v_cache.stride()[:3], page_table.stride(0)),
            (requests, page_table.shape[1], k_cache.shape[0], k_cache.shape[1]))


def rotary_append(q, k, v, inv_freq, k_cache, v_cache, page_table, lengths, cu_seqlens=None, *, interleaved=False,
                  amplitude=1.0, out=None, device_status=None, stream=None):
    """Rotary positions on the queries and keys of new tokens; keys and values go to their pages.

    q [batch, window, H, dim], k and v [batch, window, G, dim] (or without the window
    dimension, one token each), or packed [tokens, ...] with cu_seqlens [batch + 1].
    lengths [batch] int32 counts each request's tokens, the new ones, its last, among them.
    Token i of request b lies in row i mod page_size of page page_table[b, i // page_size] of
    k_cache and v_cache [pages, page_size, G, dim].  inv_freq [n] fp32 turns the first
    2 n columns of a head: pairs (j, j + n), or neighbours where `interleaved`;
    amplitude multiplies sines and cosines.  Returns the turned queries, shaped like q;
    out may be q.  A request of length 0 is skipped, its rows are zero.
    """
    lib = _lib or _load()
    if stream is None and out is None and device_status is None:
        r = _calls.rotary(q, k, v, inv_freq, k_cache, v_cache, page_table, lengths, cu_seqlens, interleaved, amplitude)
        if r is not None:
            return r if type(r) is not int else _raise("rotary_append", r)
    _check_grad(q, k, v, inv_freq, k_cache, v_cache, out)
    _need(q.dtype in _INPUTS, f"q must be bfloat16 or float32, got {q.dtype}")
    n = q.dim() - 2
    _need(n == 1 or (n == 2 and cu_seqlens is None),
          "q must be [batch, window, heads, dim] or [batch, heads, dim], or [tokens, heads, dim] with cu_seqlens")
    lead, (H, dim) = tuple(q.shape[:n]), q.shape[n:]
    _need(k_cache.dim() == 4, "k_cache must be [pages, page_size, kv_heads, dim]")
    G = k_cache.shape[2]
    _check_heads(q, "q", q.dtype, lead, H, dim)
    _check_heads(k, "k", q.dtype, lead, G, dim)
    _check_heads(v, "v", q.dtype, lead, G, dim)
    _need(inv_freq.dim() == 1, "inv_freq must be a vector")
    _check_vector(inv_freq, "inv_freq", inv_freq.shape[0], _F32)
    _check_device(q, k, v, inv_freq, k_cache, v_cache, page_table, lengths, cu_seqlens, out, device_status)
    requests = q.shape[0]
    if cu_seqlens is not None:
        requests = cu_seqlens.shape[0] - 1
        _need(requests >= 0, "cu_seqlens must have at least one entry")
        _check_vector(cu_seqlens, "cu_seqlens", requests + 1, _I32)
    ptrs, strides, sizes = _pages(k_cache, v_cache, page_table, lengths, q.dtype, dim, requests)
    if out is None:
        out = _like(q, stream)
    else:
        _check_out(out, q)
        _check_heads(out, "out", q.dtype, lead, H, dim)
        need = H * dim
        for size, stride in zip(reversed(lead), reversed(out.stride()[:n])):
            _need(size < 2 or stride >= need, "rows of out overlap")
            need = max(need, size * stride)

    def both(t):  # batch and token strides
        s = t.stride()
        return (0, s[0]) if cu_seqlens is not None else (s[0], s[1] if n == 2 else 0)
    rc = lib.rsm_rotary_append(_pack_rotary(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), inv_freq.data_ptr(), _ptr(cu_seqlens), out.data_ptr(),
        _status(device_status), *ptrs, *strides, *sizes, q.shape[0] if cu_seqlens is not None else 0, *both(q), *both(k),
        *both(v), *both(out), 0 if cu_seqlens is not None else lead[1] if n == 2 else 1, H, G, dim, 2 * inv_freq.shape[0],
        _INPUTS[q.dtype], bool(interleaved), float(amplitude)), _handle(stream, q.get_device()))
    if rc != 0:
        _raise("rotary_append", rc)
    return out


def paged_attention(q, k_cache, v_cache, page_table, lengths, *, scale=None, out=None, workspace=None,
                    device_status=None, stream=None):
    """Attention of new tokens over the pages of their requests.

    q [batch, window, H, dim], or [batch, H, dim] for one token each; pages, page_table
    and lengths as for rotary_append, which has put the new tokens' keys and values in.
    New token t of request b is at position lengths[b] - window + t and sees all tokens
    up to its own; H is a multiple of the G key heads.  scale defaults to
    dim ** -0.5.  Returns the outputs, shaped like q (out may be q); rows of a request of length 0 are
    zero.  A call that may be split over the caches' length needs a workspace, which is
    allocated where `workspace` (a contiguous uint8 CUDA tensor, which belongs to one call at a time) is not given.
    """
    lib = _lib or _load()
    if stream is None and out is None and workspace is None and device_status is None:
        r = _calls.attention(q, k_cache, v_cache, page_table, lengths, scale)
        if r is not None:
            return r if type(r) is not int else _raise("paged_attention", r)
    _check_grad(q, k_cache, v_cache, out)
    _need(q.dtype in _INPUTS, f"q must be bfloat16 or float32, got {q.dtype}")
    n = q.dim() - 2
    _need(n in (1, 2), "q must be [batch, window, heads, dim] or [batch, heads, dim]")
    lead, (H, dim) = tuple(q.shape[:n]), q.shape[n:]
    _check_heads(q, "q", q.dtype, lead, H, dim)
    _check_device(q, k_cache, v_cache, page_table, lengths, out, workspace, device_status)
    _need(k_cache.dim() == 4, "k_cache must be [pages, page_size, kv_heads, dim]")
    ptrs, strides, sizes = _pages(k_cache, v_cache, page_table, lengths, q.dtype, dim, q.shape[0])
    if out is None:
        out = _like(q, stream)
    else:
        _check_out(out, q)
        _need(out.is_contiguous(), "out must be contiguous")
    args = [q.data_ptr(), out.data_ptr(), 0, _status(device_status), *ptrs, *strides, *sizes, q.stride(0),
            q.stride(1) if n == 2 else 0, 0, lead[1] if n == 2 else 1, H, k_cache.shape[2], dim, _INPUTS[q.dtype],
            dim ** -0.5 if scale is None else float(scale)]
    packed = _pack_attention(*args)
    size = lib.rsm_paged_attention_workspace(packed)
    if size < 0:
        _raise("paged_attention", size)
    if size > 0:
        if workspace is None:
            make = lambda: torch.empty(size, dtype=torch.uint8, device=q.device)  # noqa: E731
            workspace = make() if stream is None else _new_on(stream, make)
        _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(), "workspace must be a contiguous uint8 tensor")
        args[2], args[4 + 4 + 7 + 4 + 2] = workspace.data_ptr(), workspace.numel()
        packed = _pack_attention(*args)
    rc = lib.rsm_paged_attention(packed, _handle(stream, q.get_device()))
    if rc != 0:
        _raise("paged_attention", rc)
    return out


def copy_pages(page_ptrs, page_strides, src_pages, dst_pages, *, dtype, page_elements, num_pages, device_status=None,
               stream=None):
    """Page dst_pages[i] of every pool becomes page src_pages[i], for all pools in one call.

    page_ptrs and page_strides [pools] int64 are tables on the device (pointer_table and
    stride_table of the pools, [num_pages, ...] with contiguous pages), src_pages and
    dst_pages [pairs] int32; a page is page_elements elements of `dtype` (any type of a
    state or cache: pools of convolution caches and states are pages of slots too).  A
    pair with a negative page is skipped.  Destinations are distinct and no pair's source.
    """
    lib = _lib or _load()
    code = _STATES.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    if stream is None and device_status is None:
        r = _calls.copy(page_ptrs, page_strides, src_pages, dst_pages, code, page_elements, num_pages)
        if r is not None:
            return None if r == 0 else _raise("copy_pages", r)
    _need(page_ptrs.dim() == 1 and src_pages.dim() == 1, "page_ptrs and src_pages must be vectors")
    pools, pairs = page_ptrs.shape[0], src_pages.shape[0]
    _check_vector(page_ptrs, "page_ptrs", pools, torch.int64)
    _check_vector(page_strides, "page_strides", pools, torch.int64)
    _check_vector(src_pages, "src_pages", pairs, _I32)
    _check_vector(dst_pages, "dst_pages", pairs, _I32)
    _check_device(page_ptrs, page_strides, src_pages, dst_pages, device_status)
    page_elements = int(page_elements)
    _need(abs(page_elements) < 2 ** 63, f"page_elements must fit 64 bits, got {page_elements}")
    rc = lib.rsm_copy_pages(_pack_copy(
        page_ptrs.data_ptr(), page_strides.data_ptr(), src_pages.data_ptr(), dst_pages.data_ptr(), _status(device_status),
        page_elements, pools, pairs, _int32(num_pages, "num_pages"), code), _handle(stream, page_ptrs.get_device()))
    if rc != 0:
        _raise("copy_pages", rc)


def rotary_frequencies(rotary_dim, base=10000.0, *, scaling=None, factor=1.0, original_length=None, slow=1.0, fast=32.0,
                       device=None):
    """(inv_freq, amplitude) for rotary_append: base ** (-2 j / rotary_dim), scaled for contexts `factor` times longer.

    scaling None: as they are; "linear": all divided by factor; "ntk": a base that divides the
    lowest by factor and leaves the highest; "yarn" (Peng et al., 2023): a frequency that makes fewer
    than `slow` turns over original_length tokens is divided by factor, one that makes more
    than `fast` is left, one with r turns between is mixed by the paper's equation, keep f + (1 - keep) f / factor
    with keep = (r - slow) / (fast - slow), linear in r, and the amplitude is 0.1 ln(factor) + 1.  Programs that take
    `keep` as linear in the pair's index j instead, between rounded bounds, get other frequencies there: a model that
    was trained so needs those, which go to rotary_append as any vector does.
    """
    _need(rotary_dim > 0 and rotary_dim % 2 == 0, "rotary_dim must be even and positive")
    _need(factor > 0, "factor must be positive")
    _need(base > 0, "base must be positive")
    _need(scaling in (None, "linear", "ntk", "yarn"), f"unknown scaling {scaling!r}")
    if scaling == "ntk":
        _need(rotary_dim > 2, "ntk scaling needs a rotary_dim above 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        _need(original_length is not None and original_length > 0, "yarn scaling needs original_length, which is positive")
        _need(fast > slow, "fast must be above slow")
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return f.to(device=device or "cuda", dtype=_F32), amplitude
