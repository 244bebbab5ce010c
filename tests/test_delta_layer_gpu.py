"""GatedDeltaNorm as a layer calls it (GPU): every input a slice of one projection, gradients back
into the projection, and rows behind the last sequence.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn

HK, HV, K, V = 2, 4, 64, 128
WIDTHS = (HK * K, HK * K, HV * V, HV * V)
SHAPES = ((HK, K), (HK, K), (HV, V), (HV, V))


def slices(wide, lead):
    """q, k, v and the gate as columns of one tensor."""
    return [t.unflatten(-1, s) for t, s in zip(wide.split(WIDTHS, -1), SHAPES)]


def inputs(*lead):
    gen = torch.Generator(device="cuda").manual_seed(len(lead))
    wide = 0.2 * torch.randn(*lead, sum(WIDTHS), generator=gen, device="cuda")
    g = -torch.rand(*lead, HV, generator=gen, device="cuda")
    beta = torch.rand(*lead, HV, generator=gen, device="cuda")
    return wide.bfloat16(), g, beta


@pytest.mark.parametrize("lead", [(70,), (3, 37)])
def test_slices_of_one_projection(lead):
    mod = gn.GatedDeltaNorm(V, dtype=torch.float32, device="cuda")
    wide, g, beta = inputs(*lead)
    out, grads = [], []
    for copy in (False, True):
        w = wide.clone().requires_grad_()
        q, k, v, gate = (t.contiguous() if copy else t for t in slices(w, lead))
        assert copy or not gate.is_contiguous()
        y, state = mod(q, k, v, g, beta, gate)
        assert y.shape == lead + (HV, V)
        mod.weight.grad = None
        (y.float().square().sum() + state.sum()).backward()
        out.append((y, state))
        grads.append((w.grad, mod.weight.grad))
    for a, b in zip(out[0] + grads[0], out[1] + grads[1]):
        assert torch.equal(a, b)


def test_the_step_takes_slices():
    mod = gn.GatedDeltaNorm(V, device="cuda")
    wide, g, beta = inputs(6)
    pool = torch.zeros(6, HV, K, V, device="cuda")
    p2 = pool.clone()
    q, k, v, gate = slices(wide, (6,))
    y = mod.step(q, k, v, g, beta, gate, pool)
    y2 = mod.step(*(t.contiguous() for t in (q, k, v)), g, beta, gate.contiguous(), p2)
    assert torch.equal(y, y2) and torch.equal(pool, p2)


def test_rows_behind_the_last_sequence():
    """Whatever is there (the gate being finite): y is zero, and no gradient changes."""
    mod = gn.GatedDeltaNorm(V, dtype=torch.float32, device="cuda")
    wide, g, beta = inputs(90)
    cu = torch.tensor([0, 50, 80], dtype=torch.int32, device="cuda")
    seen = []
    for fill in (0.0, 3e38):
        w = wide.clone()
        w[80:] = fill
        q, k, v, gate = (t.detach().requires_grad_() for t in slices(w, (90,)))
        y, _ = mod(q, k, v, g, beta, gate, cu_seqlens=cu)
        assert not y[80:].any()
        mod.weight.grad = None
        y[:80].float().square().sum().backward()
        seen.append([y, mod.weight.grad] + [t.grad for t in (q, k, v, gate)])
    for a, b in zip(*seen):
        assert torch.equal(a, b)
