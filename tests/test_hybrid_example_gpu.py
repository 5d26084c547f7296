"""The example that serves a hybrid stack with all the operators, against one prompt over the same tokens.

Both ways round activations to bf16 at the same places, some eight times a layer, each within 2^-9 of a value root mean
square over its range (2^-8 at most, uniformly: 2^-8 / sqrt(3) / sqrt(2) or so; taken as 2^-8 / sqrt(3)); what differs
between them is the order of sums, and roundings that this turns the other way, carried on by layers that neither grow
nor shrink a difference.  Five layers of eight, two ways: sqrt(2 * 40) 2^-8 / sqrt(3), about 0.020; the bound is one and
a half times that.
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ACCEPT = [[4, 2, 0], [1, 4, 4], [3, 0, 4], [4, 4, 1], [0, 2, 3]]


@pytest.mark.parametrize("layers", ["MMAMA", "AM"])
@pytest.mark.parametrize("page", [16, 5])
def test_served_in_pieces_equals_one_prompt(layers, page):
    import hybrid_decode as ex
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    make = lambda: ex.Stack(layers=layers, page=page, pages=128)  # noqa: E731
    stack = make()
    prompts, tokens = [rand(n, stack.width) for n in (37, 150, 64)], rand(3, 20, stack.width)
    outs, lengths = ex.serve(stack, prompts, tokens, (1, 33, 64), ACCEPT)
    whole = [torch.cat([p, t[:n - len(p)]]) for p, t, n in zip(prompts, tokens, lengths)]
    want = make().prompt(whole, [0] * 3)
    for r in range(3):
        assert outs[r].shape == want[r].shape
        assert float((outs[r] - want[r]).norm() / want[r].norm()) < 0.03
    # a fork answers as its original does, and neither changes what the other holds
    stack.fork(1, 0, lengths[1])
    x = rand(1, 4, stack.width).expand(3, 4, -1).contiguous()
    y = stack.draft(x, [lengths[1], lengths[1], lengths[2]], [0] * 3)
    assert torch.equal(y[0], y[1])
    x[0] = -x[0]
    again = stack.draft(x, [lengths[1], lengths[1], lengths[2]], [0] * 3)
    assert torch.equal(again[1:], y[1:]) and not torch.equal(again[0], y[0])
