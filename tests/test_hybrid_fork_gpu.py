"""Forks in the example that serves a hybrid stack: which pages are held, by how many requests, and what forks answer."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


PAGES = 96


def check_pages(stack):
    """Every page is free or held, as often as tables have it."""
    held = stack.table[stack.table >= 0].tolist()
    assert len(stack.free) + len(set(held)) == PAGES and sorted({*stack.free, *held}) == list(range(PAGES))
    assert stack.holders == [held.count(p) for p in range(PAGES)]


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("length", [48, 50, 3])
def test_forks_again_and_again(page, length):
    """Many forks onto one target, forks of forks, and a source that is a target next: the pool does not shrink, and each
    fork answers as its source does."""
    import hybrid_decode as ex
    stack = ex.Stack(layers="MA", page=page, pages=PAGES)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    stack.prompt([rand(length, stack.width) for _ in range(3)], [0] * 3)
    check_pages(stack)
    for k in range(120):
        r, to = ((0, 1), (0, 1), (1, 2), (2, 0))[k % 4]
        stack.fork(r, to, length)
        check_pages(stack)
        if k % 7 == 0:  # drafts, all rejected
            y = stack.draft(rand(1, 4, stack.width).expand(3, 4, -1).contiguous(), [length] * 3, [0] * 3)
            check_pages(stack)
            assert torch.equal(y[r], y[to])
    full = length // page
    assert len(set(stack.table[:, :full].flatten().tolist())) == full
    for r in (1, 0, 2):
        stack.release(r)
        check_pages(stack)
    assert len(stack.free) == PAGES
