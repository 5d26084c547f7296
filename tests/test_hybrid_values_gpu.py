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


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [64, 22])
@pytest.mark.parametrize("tokens", [40, 6000])
def test_rotary_frequencies_that_are_no_numbers(tokens, dim, interleaved, dtype):
    """Pairs of a frequency that is not a number, infinite or 2^40 and more become NaN, by each kernel; the others, one just
    below 2^40 among them, are as ever."""
    H, G, page, n = 3, 1, 64, 10
    table = torch.arange(-(-tokens // page), device="cuda", dtype=torch.int32)[None]
    kc, vc = base.pools(base.gen(1), table.numel(), page, G, dim, dtype, False)
    q, k, v = (base.rand(base.gen(i), tokens, h, dim, dtype=dtype) for i, h in ((2, H), (3, G), (4, G)))
    freq = base.rand(base.gen(5), n).abs()
    freq[2] = 2.0 ** 40 - 2.0 ** 17
    odd = [1, 4, 5, 8]
    freq[odd] = torch.tensor([float("nan"), float("inf"), -float("inf"), -2.0 ** 40], device="cuda")
    cu, status = i32([0, tokens]), base.word()
    got = rsm.rotary_append(q, k, v, freq, kc, vc, table, i32([tokens]), cu, interleaved=interleaved, device_status=status)
    assert int(status) == 0
    columns = [c for j in odd for c in ((2 * j, 2 * j + 1) if interleaved else (j, j + n))]
    at = torch.arange(tokens, device="cuda")
    to = table[0, at // page].long(), at % page
    keys = kc[to]
    assert bool(got[..., columns].isnan().all()) and bool(keys[..., columns].isnan().all())
    good = torch.where(freq.abs() < 2.0 ** 40, freq, 0.0)
    wq, mq = ref.rotate(q, at, good, interleaved, 1.0)
    wk, mk = ref.rotate(k, at, good, interleaved, 1.0)
    others = [c for c in range(dim) if c not in columns]
    for y, w, m in ((got, wq, mq), (keys, wk, mk)):
        base.close(y[..., others], w[..., others], (base.U[dtype] * w.abs() * 1.01 + 16 * base.E * m)[..., others])
    assert torch.equal(vc[to], v)
