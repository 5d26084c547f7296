"""Shapes at which the layer operators change their way: how many sequences are put in order, how many heads a CTA
takes, how many new tokens and ring rows there are.  Bounds and references are test_block_ops_gpu's."""
import pytest

torch = pytest.importorskip("torch")

import block_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402
import test_block_ops_gpu as base  # noqa: E402
from test_block_ops_gpu import BF16, F16, F32, i32  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

I8, F8 = torch.int8, torch.float8_e4m3fn


def ragged(n, most, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, most + 1, (n,), generator=g).tolist()


@pytest.mark.parametrize("n", [2, 31, 32, 33, 70])
@pytest.mark.parametrize("state", [F32, BF16])
def test_prefill_many_ragged_sequences(n, state):
    """Up to 32 sequences are taken longest first; equal lengths and empty ones among them."""
    lens = ragged(n, 150, n)
    lens[0] = lens[-1] = 129
    base.check_prefill(lens, 4, 2, 64, 128, BF16, state, seed=n)


@pytest.mark.parametrize("tokens", [1, 7, 8, 9, 15])
def test_prefill_few_tokens(tokens):
    base.check_prefill([tokens], 6, 2, 64, 128, BF16, F32, seed=tokens)
    base.check_prefill([1] * tokens, 6, 2, 64, 128, BF16, BF16, seed=tokens)


@pytest.mark.parametrize("lens,H,G", [([300], 200, 4), ([130, 200, 64], 152, 8), ([1100], 80, 1), ([5000, 10], 6, 2)], ids=str)
def test_prefill_heads_a_cta(lens, H, G):
    """One head a CTA, two, and few long sequences in segments."""
    base.check_prefill(lens, H, G, 64, 128, BF16, F32, seed=H)


@pytest.mark.parametrize("offset,stride", [(0, 8), (8, 16), (3, 8), (0, 5)])
def test_prefill_into_a_slice(offset, stride):
    """Outputs into columns of a wider tensor, on 16 bytes and not; its other columns stay."""
    T, H = 140, 4
    x, dt, A, B, C, D = base.tokens((T,), H, 2, 64, 128, BF16, 21)
    wide = torch.full((T, H * 64 + offset + stride), 7.0, dtype=BF16, device="cuda")
    out = wide[:, offset:offset + H * 64].unflatten(-1, (H, 64))
    y = rsm.ssm_prefill(x, dt, A, B, C, i32([0, T]), D=D, out=out)
    wy, wm, _, _ = ref.prefill(x, dt, A, B, C, [0, T], torch.zeros(1, H, 64, 128, device="cuda"), None, D)
    base.close(y, wy, 2.0 ** -8, wm, base.y_terms(BF16, T), "y")
    assert bool((wide[:, :offset] == 7).all()) and bool((wide[:, offset + H * 64:] == 7).all())


@pytest.mark.parametrize("state", [F32, BF16, F16])
@pytest.mark.parametrize("T", [2, 5, 8, 9, 16])
def test_step_several_tokens(state, T):
    base.check_step(3, T, 6, 2, 64, 128, BF16, state, False, pads=(1,), seed=T, strong=True)
    base.check_step(2, T, 3, 3, 64, 128, BF16, state, True, seed=T + 1, sliced=3, skip=False)


def test_step_many_heads_a_cta():
    base.check_step(80, 2, 128, 4, 64, 128, BF16, BF16, True, pads=(7,), seed=31)
    base.check_step(80, 1, 128, 4, 64, 128, BF16, F16, False, seed=32)


@pytest.mark.parametrize("state", [F32, BF16, F16, I8, F8])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16])
def test_decode_rings_and_new_tokens(state, T):
    base.check_decode(3, T, 64, 6, 2, 64, 128, BF16, state, lens=[64 - T, 17, 0], seed=T)
    base.check_decode(2, T, 40, 3, 3, 64, 128, BF16, state, lens=[16 - min(T, 16), 33 - T], seed=T + 1, sliced=3)


@pytest.mark.parametrize("state", [BF16, I8])
def test_decode_many_heads_a_cta(state):
    base.check_decode(80, 3, 16, 128, 4, 64, 128, BF16, state, pads=(3,), seed=41)
