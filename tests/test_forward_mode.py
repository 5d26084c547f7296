"""The operators are forward only: a tensor with a tangent of forward-mode differentiation is refused, whether gradients
are recorded or not, since no_grad() keeps tangents."""
import pytest

torch = pytest.importorskip("torch")

import torch.autograd.forward_ad as fwd  # noqa: E402

import mamba_replayssm_state_gb300 as rsm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def calls(dev):
    """Every operator that takes tensors of values: (function of the keyword arguments, those that may have a tangent,
    the others)."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s, t=BF16: torch.randn(s, generator=g).to(dev, t)  # noqa: E731
    b, T, H, G = 3, 2, 4, 2
    tokens = dict(x=r(b, T, H, 64), dt=r(b, T, H, t=F32).abs(), A=-r(H, t=F32).abs(), B=r(b, T, G, 128), C=r(b, T, G, 128), D=r(H, t=F32))
    packed = {k: v.flatten(0, 1) if v.dim() > 1 else v for k, v in tokens.items()}
    state, three, zero = r(b, H, 64, 128, t=F32), i32([0, 1, 2], dev), i32([0, 0, 0], dev)
    ring = dict(x_cache=r(b, 8, H, 64), B_cache=r(b, 8, G, 128), dt_cache=r(b, 8, H, t=F32))
    rows = dict(x=r(4, 64, t=F32), weight=r(64, t=F32))
    conv = dict(weight=r(264, 4, t=F32), bias=r(264, t=F32), cache=r(b, 6, 264))
    pages = dict(k_cache=r(6, 16, G, 64), v_cache=r(6, 16, G, 64))
    where = dict(page_table=i32([[0, 1], [2, 3], [4, 5]], dev), lengths=i32([20, 3, 31], dev))
    return {
        "ssm_prefill": (rsm.ssm_prefill, packed, dict(cu_seqlens=i32([0, 6], dev))),
        "ssm_step": (rsm.ssm_step, dict(state=state, **tokens), dict(slots=three)),
        "replayssm_decode": (rsm.replayssm_decode, dict(state=state, **ring, **tokens),
                             dict(slots=three, ring_start=zero, ring_len=zero)),
        "add_rms_norm": (lambda **k: rsm.add_rms_norm(**k)[0], dict(residual=r(4, 64, t=F32), **rows), {}),
        "gated_rms_norm": (rsm.gated_rms_norm, dict(z=r(4, 64, t=F32), **rows), {}),
        "causal_conv": (rsm.causal_conv, dict(x=r(9, 264), **conv), dict(cu_seqlens=i32([0, 2, 5, 9], dev), slots=three)),
        "causal_conv_step": (rsm.causal_conv_step, dict(x=r(b, T, 264), **conv), dict(slots=three, positions=zero)),
        "rotary_append": (rsm.rotary_append, dict(q=r(b, T, H, 64), k=r(b, T, G, 64), v=r(b, T, G, 64), inv_freq=r(32, t=F32), **pages), where),
        "paged_attention": (rsm.paged_attention, dict(q=r(b, T, H, 64), **pages), where)}


NAMES = ["ssm_prefill", "ssm_step", "replayssm_decode", "add_rms_norm", "gated_rms_norm", "causal_conv", "causal_conv_step",
         "rotary_append", "paged_attention"]


def refused(f, values, others, ways):
    with fwd.dual_level():
        for name, t in values.items():
            args = values | {name: fwd.make_dual(t.clone(), torch.ones_like(t))}
            for way in ways:
                with pytest.raises(ValueError, match="has a tangent"):
                    f(**args, **others, **way)
                with torch.no_grad(), pytest.raises(ValueError, match="has a tangent"):
                    f(**args, **others, **way)


@pytest.mark.parametrize("name", NAMES)
def test_a_tangent_is_refused_before_any_other_check(name):
    f, values, others = calls("cpu")[name]
    refused(f, values, others, [{}])
    with fwd.dual_level(), pytest.raises(ValueError, match="CUDA"):
        f(**values, **others)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("name", NAMES)
def test_a_tangent_is_refused_by_either_way_into_the_library(name):
    """Results allocated (the C++ side's call) or passed; tensors without one are served within a dual level as outside."""
    f, values, others = calls("cuda")[name]
    fresh = lambda: {k: v.clone() for k, v in values.items()}  # noqa: E731
    want = f(**fresh(), **others)
    refused(f, fresh(), others, [{}, {"out": torch.empty_like(want)}])
    with fwd.dual_level():
        assert torch.equal(f(**fresh(), **others), want)
        primal = {k: fwd.unpack_dual(fwd.make_dual(v, v)).primal if v.is_floating_point() else v for k, v in fresh().items()}
        assert torch.equal(f(**primal, **others), want)
