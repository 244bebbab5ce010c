"""Gradients that autograd hands over as views at any offset of a flat buffer, as the backward of a
concatenation does: the same result as from a tensor of their own (GPU).
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn


def behind_one(t):
    """t's values behind one other in a flat tensor: its gradient starts one element in."""
    return torch.cat([torch.zeros(1, dtype=t.dtype, device=t.device), t.flatten()])


def both(outputs, leaves):
    """The leaves' gradients from the outputs' squares, directly and through flat buffers."""
    got = []
    for wrap in (lambda t: t, behind_one):
        loss = sum(wrap(t).float().square().sum() for t in outputs())
        got.append(torch.autograd.grad(loss, leaves))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def rand(*shape, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype).requires_grad_()


def test_gated_norm():
    x, g, w = rand(9, 64), rand(9, 64), rand(64)
    both(lambda: [gn.gated_rmsnorm(x, g, w)], [x, g, w])


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_block_norm(res):
    a, r, g, w1, w2 = rand(9, 64), rand(9, 64, dtype=res), rand(9, 64), rand(64), rand(64)
    both(lambda: gn.block_rmsnorm(a, r, w1, w2, g=g), [a, r, g, w1, w2])


def test_delta_rule():
    q, k, v = rand(70, 1, 64), torch.nn.functional.normalize(rand(70, 1, 64), dim=-1).detach(), rand(70, 2, 64)
    beta = torch.rand(70, 2, device="cuda").requires_grad_()
    g = (-torch.rand(70, 2, device="cuda")).requires_grad_()
    both(lambda: gn.gated_delta_rule(q, k, v, g, beta), [q, v, g, beta])
