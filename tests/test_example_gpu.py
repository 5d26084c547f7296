"""The example that serves a stack of layers with all the operators, against one prompt over the same tokens.

Both ways round activations to bf16 at the same places, some ten times a layer, each within 2^-9 of a value (root
mean square over its range: 2^-9 / sqrt(3)); a rounding that differs is a difference of that size, carried on by
layers that neither grow nor shrink it.  Four layers of ten: sqrt(2 * 40) 2^-9 / sqrt(3), about 0.010; the bound is
twice that.
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_served_in_pieces_equals_one_prompt(state):
    import speculative_decode as ex
    stack = ex.Stack(layers=4, width=512, heads=16, groups=2, requests=3, ring=8, state_dtype=state)
    g = torch.Generator(device="cuda").manual_seed(9)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    prompts, tokens = [rand(k, stack.width) for k in (1, 129, 40)], rand(3, 19, stack.width)
    outs = ex.serve(stack, prompts, tokens, accept=[[4, 0, 2], [3, 4, 1], [0, 2, 4]])
    whole = [torch.cat([p, t]) for p, t in zip(prompts, tokens)]
    cu = torch.tensor([0] + [len(w) for w in whole], device="cuda").cumsum(0, dtype=torch.int32)
    want = stack.prompt(torch.cat(whole), cu, torch.arange(3, dtype=torch.int32, device="cuda"))
    for r in range(3):
        w = want[cu[r]:cu[r + 1]]
        assert outs[r].shape == w.shape
        # a bf16 checkpoint is rounded at every commit, each within 2^-9 of the state: as many roundings again
        assert float((outs[r] - w).norm() / w.norm()) < (0.02 if state == torch.float32 else 0.03)
