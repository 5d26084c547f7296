"""The layer operators without a GPU: struct layouts, and what the C ABI and
the Python entry points refuse before any CUDA call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import mamba_replayssm_state_gb300 as rsm  # noqa: E402
from mamba_replayssm_state_gb300 import block  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    return block._load()


def call(fn, a):
    return fn(bytes(a), None)


def test_struct_layouts(lib):
    for i, cls in enumerate(block.ARGS):
        assert lib.rsm_block_args_size(i) == ctypes.sizeof(cls)
    assert lib.rsm_block_args_size(5) == 0 and lib.rsm_block_args_size(-1) == 0


def test_package_exposes_the_operators():
    for n in ("ssm_prefill", "ssm_step", "replayssm_decode", "add_rms_norm", "gated_rms_norm"):
        assert callable(getattr(rsm, n)) and n in rsm.__all__


def common(a):
    for f in ("x", "B", "C", "dt", "A", "out", "state"):
        setattr(a, f, 0x10000)
    a.num_slots, a.num_heads, a.num_groups, a.dim, a.dstate = 8, 16, 2, 64, 128
    a.state_dtype, a.input_dtype, a.pad_slot_id = rsm.RSM_F32, rsm.RSM_BF16, -1
    return a


def prefill_args():
    a = common(block.SsmPrefillArgs())
    a.cu_seqlens = 0x10000
    a.tokens, a.num_seqs = 100, 2
    return a


def step_args():
    a = common(block.SsmStepArgs())
    a.src_slots, a.batch, a.window = 0x10000, 4, 1
    return a


def decode_args():
    a = common(block.ReplaySsmDecodeArgs())
    for f in ("x_cache", "B_cache", "dt_cache", "slots", "ring_start", "ring_len"):
        setattr(a, f, 0x10000)
    a.batch, a.window, a.ring_buffer_len = 4, 1, 8
    return a


SHARED = [("x", None, -1, "x is NULL"), ("dt", None, -1, "dt is NULL"), ("A", None, -1, "A is NULL"),
          ("out", None, -1, "out is NULL"), ("num_groups", 3, -1, "num_groups"), ("num_heads", 0, -1, "num_groups"),
          ("dim", 0, -1, "positive"), ("dstate", 96, -2, "no kernel"), ("num_slots", -1, -1, "num_slots"),
          ("input_dtype", rsm.RSM_F16, -1, "input_dtype"), ("state_dtype", 9, -1, "state_dtype")]
REFUSALS = (
    [("rsm_ssm_prefill", prefill_args, *r) for r in SHARED] + [("rsm_ssm_step", step_args, *r) for r in SHARED] +
    [("rsm_replayssm_decode", decode_args, *r) for r in SHARED] +
    [("rsm_ssm_prefill", prefill_args, *r) for r in [
        ("cu_seqlens", None, -1, "cu_seqlens"), ("num_seqs", -1, -1, "num_seqs"), ("tokens", -1, -1, "tokens"),
        ("state_dtype", rsm.RSM_I8, -1, "state_dtype")]] +
    [("rsm_ssm_step", step_args, *r) for r in [
        ("src_slots", None, -1, "src_slots"), ("state", None, -1, "state is NULL"), ("window", 0, -1, "window"),
        ("batch", -1, -1, "batch"), ("state_dtype", rsm.RSM_FP8_E4M3, -1, "one-byte")]] +
    [("rsm_replayssm_decode", decode_args, *r) for r in [
        ("slots", None, -1, "slots"), ("ring_start", None, -1, "ring_start"), ("x_cache", None, -1, "x_cache"),
        ("ring_buffer_len", 0, -1, "ring_buffer_len"), ("window", 9, -1, "window"),
        ("state_dtype", rsm.RSM_I8, -1, "state_scale")]])


@pytest.mark.parametrize("name,make,field,value,code,msg", REFUSALS, ids=[f"{r[0][4:]}-{r[2]}-{r[3]}" for r in REFUSALS])
def test_refusals(lib, name, make, field, value, code, msg):
    a = make()
    setattr(a, field, value)
    assert call(getattr(lib, name), a) == code
    assert msg in lib.rsm_block_last_error().decode()


def test_slots_without_a_pool_are_refused(lib):
    a = prefill_args()
    a.state, a.final_slots = None, 0x10000
    assert call(lib.rsm_ssm_prefill, a) == -1 and "state is NULL" in lib.rsm_block_last_error().decode()


def test_one_byte_states_are_64_by_128(lib):
    a = decode_args()
    a.state_dtype, a.dstate, a.state_scale = rsm.RSM_I8, 64, 0x10000
    assert call(lib.rsm_replayssm_decode, a) == -1 and "one-byte" in lib.rsm_block_last_error().decode()


def test_empty_calls_enqueue_nothing(lib):
    a = prefill_args()
    a.num_seqs = a.tokens = 0
    assert call(lib.rsm_ssm_prefill, a) == 0
    for make, fn in ((step_args, lib.rsm_ssm_step), (decode_args, lib.rsm_replayssm_decode)):
        a = make()
        a.batch = 0
        assert call(fn, a) == 0
    assert lib.rsm_block_last_error() == b""


def norm_args(cls):
    a = cls()
    for f in ("x", "weight", "out"):
        setattr(a, f, 0x10000)
    if cls is block.AddRmsNormArgs:
        a.residual = a.residual_out = 0x10000
        a.residual_dtype = rsm.RSM_F32
    else:
        a.z, a.group_size = 0x10000, 64
    a.rows, a.dim, a.input_dtype, a.eps = 2, 128, rsm.RSM_BF16, 1e-5
    return a


@pytest.mark.parametrize("cls,field,value,msg", [
    (block.AddRmsNormArgs, "x", None, "x is NULL"), (block.AddRmsNormArgs, "residual_out", None, "residual_out"),
    (block.AddRmsNormArgs, "weight", None, "weight"), (block.AddRmsNormArgs, "rows", -1, "rows"),
    (block.AddRmsNormArgs, "dim", 0, "dim"), (block.AddRmsNormArgs, "residual_dtype", rsm.RSM_F16, "residual_dtype"),
    (block.GatedRmsNormArgs, "z", None, "z is NULL"), (block.GatedRmsNormArgs, "group_size", 48, "group_size"),
    (block.GatedRmsNormArgs, "group_size", 0, "group_size"), (block.GatedRmsNormArgs, "input_dtype", 7, "input_dtype"),
    (block.GatedRmsNormArgs, "rows", -2, "rows")])
def test_norm_refusals(lib, cls, field, value, msg):
    a = norm_args(cls)
    setattr(a, field, value)
    fn = lib.rsm_add_rms_norm if cls is block.AddRmsNormArgs else lib.rsm_gated_rms_norm
    assert call(fn, a) == -1 and msg in lib.rsm_block_last_error().decode()


def test_norms_of_no_rows_enqueue_nothing(lib):
    for cls, fn in ((block.AddRmsNormArgs, lib.rsm_add_rms_norm), (block.GatedRmsNormArgs, lib.rsm_gated_rms_norm)):
        a = norm_args(cls)
        a.rows = 0
        assert call(fn, a) == 0


def test_null_args(lib):
    for f in ("rsm_ssm_prefill", "rsm_ssm_step", "rsm_replayssm_decode", "rsm_add_rms_norm", "rsm_gated_rms_norm"):
        assert getattr(lib, f)(None, None) == -1


# ----------------------------------------------------------------------------
# the Python entry points: host tensors and wrong shapes
# ----------------------------------------------------------------------------

def token_tensors(*lead, H=4, G=2, dim=64, N=128, dtype=torch.bfloat16):
    return (torch.zeros(*lead, H, dim, dtype=dtype), torch.zeros(*lead, H), torch.zeros(H),
            torch.zeros(*lead, G, N, dtype=dtype), torch.zeros(*lead, G, N, dtype=dtype))


def test_host_tensors_are_refused():
    x, dt, A, B, C = token_tensors(5)
    with pytest.raises(ValueError, match="CUDA"):
        rsm.ssm_prefill(x, dt, A, B, C, torch.tensor([0, 5], dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        rsm.add_rms_norm(torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        rsm.gated_rms_norm(torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(8))


@pytest.mark.parametrize("change,msg", [
    (dict(x=torch.zeros(5, 4, 64, dtype=torch.float16)), "bfloat16 or float32"),
    (dict(dt=torch.zeros(5, 3)), "dt must be"), (dict(dt=torch.zeros(5, 4, dtype=torch.bfloat16)), "dt must be"),
    (dict(A=torch.zeros(3)), "A must be"), (dict(C=torch.zeros(5, 2, 64, dtype=torch.bfloat16)), "C must be"),
    (dict(B=torch.zeros(5, 2, 128)), "B must be"), (dict(D=torch.zeros(5)), "D must be"),
    (dict(x=torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "contiguous")])
def test_shapes_are_checked(change, msg):
    x, dt, A, B, C = token_tensors(5)
    t = dict(x=x, dt=dt, A=A, B=B, C=C, D=None) | change
    with pytest.raises(ValueError, match=msg):
        rsm.ssm_prefill(t["x"], t["dt"], t["A"], t["B"], t["C"], torch.tensor([0, 5], dtype=torch.int32), D=t["D"])
