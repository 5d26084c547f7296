"""The operators of hybrid stacks without a GPU: struct layouts, what the C ABI and the Python entry points refuse
before any CUDA call, and the frequencies."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import mamba_replayssm_state_gb300 as rsm  # noqa: E402
from mamba_replayssm_state_gb300 import hybrid  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return hybrid._load()


def test_struct_layouts(lib):
    for i, cls in enumerate(hybrid.ARGS):
        assert lib.rsm_hybrid_args_size(i) == ctypes.sizeof(cls)
    assert lib.rsm_hybrid_args_size(5) == 0 and lib.rsm_hybrid_args_size(-1) == 0


def test_package_exposes_the_operators():
    for n in hybrid.__all__:
        assert getattr(rsm, n) is getattr(hybrid, n) and n in rsm.__all__


def filled(cls, names, **values):
    a = cls()
    for f in names.split():
        setattr(a, f, 0x10000)
    for f, v in values.items():
        setattr(a, f, v)
    return a


MOST = 2 ** 30  # of what the kernels count in 32 bits
PAGES = dict(table_width=4, num_pages=9, page_size=16, requests=2)


def conv_args():
    return filled(hybrid.CausalConvArgs, "x weight bias cu_seqlens cache slots positions", out=0x20000, tokens=9, num_seqs=2,
                  num_slots=3, channels=64, width=4, cache_rows=3, input_dtype=rsm.RSM_BF16, pad_slot_id=-1)


def step_args():
    return filled(hybrid.CausalConvStepArgs, "x weight bias cache slots positions", out=0x20000, batch=2, window=2,
                  num_slots=3, channels=64, width=4, cache_rows=5, input_dtype=rsm.RSM_BF16, pad_slot_id=-1)


def rotary_args():
    return filled(hybrid.RotaryAppendArgs, "q k v inv_freq q_out k_pages v_pages page_table lengths", window=1, num_heads=4,
                  num_kv_heads=2, dim=64, rotary_dim=64, input_dtype=rsm.RSM_BF16, amplitude=1.0, **PAGES)


def attention_args():
    return filled(hybrid.PagedAttentionArgs, "q out k_pages v_pages page_table lengths", window=1, num_heads=4, num_kv_heads=2,
                  dim=64, input_dtype=rsm.RSM_BF16, scale=1.0, **PAGES)


def copy_args():
    return filled(hybrid.CopyPagesArgs, "page_ptrs page_strides src_pages dst_pages", page_elements=64, num_pools=2,
                  num_pairs=2, num_pages=9, dtype=rsm.RSM_BF16)


CONV = [("x", None, -1, "x is NULL"), ("weight", None, -1, "weight is NULL"), ("out", None, -1, "out is NULL"),
        ("channels", 0, -1, "channels"), ("width", 1, -2, "width"), ("width", 5, -2, "width"),
        ("input_dtype", rsm.RSM_F16, -1, "input_dtype"), ("num_slots", -1, -1, "num_slots"), ("cache_rows", 2, -1, "cache_rows"),
        ("slots", None, -1, "slots"), ("out", 0x10000, -1, "out must not be x")]
HEADS = [("q", None, -1, "q is NULL"), ("k_pages", None, -1, "k pages"), ("v_pages", None, -1, "v pages"),
         ("page_table", None, -1, "page_table"), ("lengths", None, -1, "lengths"), ("num_kv_heads", 3, -1, "num_kv_heads"),
         ("num_heads", 0, -1, "num_kv_heads"), ("dim", 0, -1, "dim"), ("dim", 257, -2, "at most 256"),
         ("input_dtype", rsm.RSM_I8, -1, "input_dtype"), ("requests", -1, -1, "requests"), ("page_size", 0, -1, "page_size"),
         ("num_pages", -1, -1, "num_pages"), ("table_width", -1, -1, "table_width"), ("window", 0, -1, "window")]
REFUSALS = (
    [("rsm_causal_conv", conv_args, *r) for r in CONV + [
        ("cu_seqlens", None, -1, "cu_seqlens"), ("num_seqs", -1, -1, "num_seqs"), ("tokens", -1, -1, "tokens"),
        ("cache", None, -1, "go together")]] +
    [("rsm_causal_conv_step", step_args, *r) for r in CONV + [
        ("cache", None, -1, "cache is NULL"), ("positions", None, -1, "positions"), ("cache_rows", 4, -1, "window"),
        ("window", 2 ** 31 - 1, -1, "cache_rows"), ("batch", -1, -1, "batch"), ("window", 0, -1, "window")]] +
    [("rsm_rotary_append", rotary_args, *r) for r in HEADS + [
        ("k", None, -1, "k is NULL"), ("v", None, -1, "v is NULL"), ("inv_freq", None, -1, "inv_freq"),
        ("q_out", None, -1, "q_out"), ("rotary_dim", 66, -1, "rotary_dim"), ("rotary_dim", 7, -1, "rotary_dim"),
        ("rotary_dim", -2, -1, "rotary_dim")]] +
    [("rsm_paged_attention", attention_args, *r) for r in HEADS + [("out", None, -1, "out is NULL")]] +
    [("rsm_copy_pages", copy_args, *r) for r in [
        ("page_ptrs", None, -1, "page_ptrs"), ("page_strides", None, -1, "page_strides"), ("src_pages", None, -1, "src_pages"),
        ("dst_pages", None, -1, "dst_pages"), ("page_elements", 0, -1, "page_elements"), ("page_elements", 2 ** 62, -1, "2^40"),
        ("num_pools", -1, -1, "num_pools"), ("num_pairs", -1, -1, "num_pairs"), ("num_pages", -1, -1, "num_pages"),
        ("num_pools", 2 ** 31 - 1, -1, "blocks"), ("dtype", 5, -1, "dtype"), ("dtype", -1, -1, "dtype")]])


@pytest.mark.parametrize("name,make,fields,msg", [
    ("rsm_causal_conv", conv_args, dict(num_seqs=MOST + 1), "num_seqs"),
    ("rsm_causal_conv_step", step_args, dict(window=MOST + 1, cache_rows=2 ** 31 - 1), "window"),
    ("rsm_rotary_append", rotary_args, dict(requests=MOST + 1), "requests"),
    ("rsm_rotary_append", rotary_args, dict(window=MOST + 1), "window"),
    ("rsm_rotary_append", rotary_args, dict(num_heads=2 ** 24), "a token's values"),
    ("rsm_paged_attention", attention_args, dict(requests=MOST + 1), "requests"),
    ("rsm_paged_attention", attention_args, dict(window=MOST // 4 + 1), "num_heads"),
    ("rsm_paged_attention", attention_args, dict(num_heads=2 ** 31 - 2, window=2 ** 31 - 1), "num_heads")])
def test_sizes_past_32_bits_are_refused(lib, name, make, fields, msg):
    a = make()
    for f, v in fields.items():
        setattr(a, f, v)
    assert getattr(lib, name)(bytes(a), None) == -2
    assert msg in lib.rsm_hybrid_last_error().decode() and "2^30" in lib.rsm_hybrid_last_error().decode()


@pytest.mark.parametrize("name,make,field,value,code,msg", REFUSALS,
                         ids=[f"{r[0][4:]}-{r[2]}-{r[3]}" for r in REFUSALS])
def test_refusals(lib, name, make, field, value, code, msg):
    a = make()
    setattr(a, field, value)
    assert getattr(lib, name)(bytes(a), None) == code
    assert msg in lib.rsm_hybrid_last_error().decode()


def test_positions_need_a_cache(lib):
    a = conv_args()
    a.cache = a.slots = None
    assert lib.rsm_causal_conv(bytes(a), None) == -1 and "positions" in lib.rsm_hybrid_last_error().decode()


def test_workspace_checks_sizes_only(lib):
    a = attention_args()
    a.q = a.out = a.k_pages = a.lengths = None
    a.dim = 300
    assert lib.rsm_paged_attention_workspace(bytes(a)) == -2


@pytest.mark.parametrize("name,make,field", [
    ("rsm_causal_conv", conv_args, "num_seqs"), ("rsm_causal_conv", conv_args, "tokens"),
    ("rsm_causal_conv_step", step_args, "batch"), ("rsm_rotary_append", rotary_args, "requests"),
    ("rsm_paged_attention", attention_args, "requests"), ("rsm_copy_pages", copy_args, "num_pools"),
    ("rsm_copy_pages", copy_args, "num_pairs")])
def test_empty_calls_enqueue_nothing(lib, name, make, field):
    a = make()
    setattr(a, field, 0)
    assert getattr(lib, name)(bytes(a), None) == 0 and lib.rsm_hybrid_last_error() == b""


def test_null_args(lib):
    for f in ("rsm_causal_conv", "rsm_causal_conv_step", "rsm_rotary_append", "rsm_paged_attention", "rsm_copy_pages"):
        assert getattr(lib, f)(None, None) == -1


# ----------------------------------------------------------------------------
# the Python entry points: host tensors and wrong shapes
# ----------------------------------------------------------------------------

def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


F32 = torch.float32
CALLS = {
    "causal_conv": dict(x=z(5, 8), weight=z(8, 4, dtype=F32), cu_seqlens=i32(0, 5), bias=z(8, dtype=F32), cache=z(2, 4, 8),
                        slots=i32(0), positions=i32(0)),
    "causal_conv_step": dict(x=z(1, 2, 8), weight=z(8, 4, dtype=F32), cache=z(2, 5, 8), slots=i32(0), positions=i32(0)),
    "rotary_append": dict(q=z(2, 4, 8), k=z(2, 2, 8), v=z(2, 2, 8), inv_freq=z(4, dtype=F32), k_cache=z(3, 16, 2, 8),
                          v_cache=z(3, 16, 2, 8), page_table=i32(0, 1).view(2, 1), lengths=i32(1, 1)),
    "paged_attention": dict(q=z(2, 4, 8), k_cache=z(3, 16, 2, 8), v_cache=z(3, 16, 2, 8), page_table=i32(0, 1).view(2, 1),
                            lengths=i32(1, 1)),
    "copy_pages": dict(page_ptrs=torch.zeros(2, dtype=torch.int64), page_strides=torch.zeros(2, dtype=torch.int64),
                       src_pages=i32(0), dst_pages=i32(1), dtype=BF16, page_elements=8, num_pages=3)}


@pytest.mark.parametrize("name", list(CALLS))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA"):
        getattr(rsm, name)(**CALLS[name])


@pytest.mark.parametrize("name,change,msg", [
    ("causal_conv", dict(x=z(5, 8, dtype=torch.float16)), "bfloat16 or float32"), ("causal_conv", dict(x=z(5, 8, 1)), "x must be"),
    ("causal_conv", dict(x=z(8, 5).t()), "contiguous"), ("causal_conv", dict(weight=z(8, 4)), "weight must be"),
    ("causal_conv", dict(weight=z(4, 8, dtype=F32).t()), "weight must be"), ("causal_conv", dict(bias=z(7, dtype=F32)), "bias must be"),
    ("causal_conv_step", dict(x=z(8)), "x must be"), ("causal_conv_step", dict(x=z(1, 2, 0)), "channels"),
    ("rotary_append", dict(q=z(2, 4, 8, dtype=torch.float16)), "bfloat16 or float32"), ("rotary_append", dict(q=z(4, 8)), "q must be"),
    ("rotary_append", dict(q=z(2, 1, 4, 8), cu_seqlens=i32(0, 1, 2)), "q must be"),
    ("rotary_append", dict(k=z(2, 3, 8)), "k must be"), ("rotary_append", dict(v=z(2, 2, 8, dtype=F32)), "v must be"),
    ("rotary_append", dict(q=z(2, 8, 4).transpose(1, 2)), "contiguous"), ("rotary_append", dict(inv_freq=z(4)), "inv_freq must be"),
    ("paged_attention", dict(q=z(2, 4, 8, dtype=torch.float16)), "bfloat16 or float32"),
    ("paged_attention", dict(q=z(4, 8)), "q must be"), ("paged_attention", dict(q=z(2, 8, 4).transpose(1, 2)), "contiguous"),
    ("copy_pages", dict(page_ptrs=z(2, dtype=torch.int32)), "page_ptrs must be"), ("copy_pages", dict(dst_pages=i32(1, 2)), "dst_pages must be"),
    ("copy_pages", dict(dtype=torch.float64), "unsupported dtype")])
def test_shapes_are_checked(name, change, msg):
    with pytest.raises(ValueError, match=msg):
        getattr(rsm, name)(**(CALLS[name] | change))


@pytest.mark.parametrize("name,arg", [("causal_conv", "x"), ("causal_conv", "weight"), ("causal_conv_step", "cache"),
                                      ("rotary_append", "k"), ("paged_attention", "v_cache")])
def test_gradients_are_refused(name, arg):
    t = CALLS[name][arg].clone().requires_grad_()
    with pytest.raises(ValueError, match="forward only"):
        getattr(rsm, name)(**(CALLS[name] | {arg: t}))
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        getattr(rsm, name)(**(CALLS[name] | {arg: t}))


# ----------------------------------------------------------------------------
# frequencies
# ----------------------------------------------------------------------------

def test_frequencies():
    f, a = rsm.rotary_frequencies(8, 10000.0, device="cpu")
    assert a == 1.0 and f.dtype == F32
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001]), rtol=1e-6)
    g, _ = rsm.rotary_frequencies(8, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(g, f / 4, rtol=1e-6)
    g, _ = rsm.rotary_frequencies(8, 10000.0, scaling="ntk", factor=4.0, device="cpu")
    assert float(g[0]) == 1.0 and abs(float(g[-1] / f[-1]) - 0.25) < 1e-6


def test_frequencies_yarn():
    L, s = 4096, 16.0
    f, _ = rsm.rotary_frequencies(128, device="cpu")
    g, a = rsm.rotary_frequencies(128, scaling="yarn", factor=s, original_length=L, device="cpu")
    assert abs(a - (0.1 * math.log(s) + 1)) < 1e-12
    turns = L * f.double() / (2 * math.pi)
    ratio = (g / f).double()
    assert torch.allclose(ratio[turns >= 32], torch.ones(1, dtype=torch.float64), rtol=1e-6)
    assert torch.allclose(ratio[turns <= 1], torch.full((1,), 1 / s, dtype=torch.float64), rtol=1e-6)
    between = (turns > 1) & (turns < 32)
    mix = (turns - 1) / 31
    assert torch.allclose(ratio[between], (mix + (1 - mix) / s)[between], rtol=1e-5) and int(between.sum()) > 10


@pytest.mark.parametrize("kw,msg", [(dict(slow=4.0, fast=4.0), "above slow"), (dict(original_length=0), "positive"),
                                    (dict(base=0.0), "base")])
def test_frequencies_that_are_no_numbers_are_refused(kw, msg):
    with pytest.raises(ValueError, match=msg):
        rsm.rotary_frequencies(8, scaling="yarn", device="cpu", **(dict(original_length=4096, factor=2.0) | kw))


@pytest.mark.parametrize("args,kw,msg", [((7,), {}, "even"), ((0,), {}, "even"), ((8,), dict(scaling="other"), "unknown"),
                                         ((8,), dict(factor=0.0), "factor"), ((8,), dict(scaling="yarn"), "original_length"),
                                         ((2,), dict(scaling="ntk"), "above 2")])
def test_frequencies_refusals(args, kw, msg):
    with pytest.raises(ValueError, match=msg):
        rsm.rotary_frequencies(*args, **kw, device="cpu")
