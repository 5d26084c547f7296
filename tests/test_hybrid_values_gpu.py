"""Attention over pages where values are near the largest of their type.  Bounds and references are
test_hybrid_ops_gpu's."""
import pytest

torch = pytest.importorskip("torch")

import hybrid_reference as ref  # noqa: E402
import mamba_replayssm_state_gb300 as rsm  # noqa: E402
import test_hybrid_ops_gpu as base  # noqa: E402
from test_hybrid_ops_gpu import BF16, F32, i32  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 72), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128), (F32, 256), (BF16, 20)])
@pytest.mark.parametrize("H", [4, 32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_values_near_the_largest(sign, H, dtype, dim):
    """Scores that rise by 5.5 (2^7.9 in the weight) from tokens to later ones, all values in 2^117 .. 2^118: an output is
    no larger than its values, and no sum on the way may be infinite.  (600 values below 2^118 with weights of at most
    one sum to less than 2^127.3; with weights that rise to 2^7.9 the 75 later tokens of a warp would sum to 2^131.)"""
    lengths = [600] * 64
    q, kc, vc, table = base.attention_world(lengths, 1, H, 4, dim, 16, dtype, False, dim)
    q.zero_(), kc.clamp_(-2, 2)
    q[..., 0], kc[..., 0] = sign, 0.0
    for r in range(64):
        step = 64 if r % 2 else 16  # (tiles of 32, 64 and 128 tokens, of which a warp takes steps of 16)
        for a in range(step, 600, 2 * step):
            at = torch.arange(a, min(a + step, 600), device="cuda")
            kc[table[r, at // 16].long(), at % 16, :, 0] = 5.5 * sign
    vc = ((0.5 + 0.5 * torch.rand(vc.shape, generator=base.gen(1), device="cuda")) * 2.0 ** 118).to(dtype)
    got = rsm.paged_attention(q, kc, vc, table, i32(lengths), scale=1.0)
    assert bool(got.isfinite().all())
    base.attention_check(q, kc, vc, table, lengths, got, scale=1.0)


@pytest.mark.parametrize("H,T,dim", [(H, T, dim) for H, T in ((4, 1), (8, 4), (16, 1), (16, 2), (16, 4), (20, 4), (16, 6), (24, 4))
                                     for dim in (64, 72, 128, 256) if H // 4 * T <= (8 if dim == 256 else 24)])
def test_attention_weights_are_not_rounded_to_bf16(H, T, dim):
    """Up to 24 rows a key head (8 of heads above 128), bf16: weights are sums of two bf16 values, cut off and then rounded, so
    off by 2^-7 2^-8 at most.  Values of both signs make outputs that are small beside the sum of their terms, where
    2^-8 of each weight would show."""
    lengths = [T + n for n in (1, 7, 16, 40, 64, 90, 200, 700)]
    q, kc, vc, table = base.attention_world(lengths, T, H, 4, dim, 16, BF16, False, dim + H + T)
    got = rsm.paged_attention(q, kc, vc, table, i32(lengths))
    y, m, top = ref.attention(q, kc, vc, table, lengths, dim ** -0.5)
    exact = base.attention_bound(y, m, top, dim, max(lengths), F32) - base.U[F32] * y.abs() * 1.01
    base.close(got, y, base.U[BF16] * y.abs() * 1.01 + exact + 2.0 ** -15 * m)
