"""attention() has first gradients only: a second one raises instead of missing its part."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_second_gradient_raises(cuda_device, fa2_lib):
    g = torch.Generator().manual_seed(0)
    leaves = [torch.randn(1, 2, 70, 64, generator=g).to(torch.bfloat16).cuda().requires_grad_() for _ in range(3)]
    o = lambda: fa2_lib.attention(*leaves, causal=True).float()  # noqa: E731
    # gradients of o that are constants, and some that want a gradient
    for loss in (lambda: o().sum(), lambda: o().square().sum()):
        want = torch.autograd.grad(loss(), leaves)
        got = torch.autograd.grad(loss(), leaves, create_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for t in leaves:  # beside a term that can be differentiated
            with pytest.raises(RuntimeError, match="differentiated"):
                torch.autograd.grad(got[0].float().square().sum() + t.float().square().sum(), t, retain_graph=True)
    # without create_graph gradients are as ever
    o().sum().backward()
    assert all(t.grad is not None and not t.grad.requires_grad for t in leaves)
