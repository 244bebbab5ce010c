"""BlockRMSNorm after the casts that a model goes through (GPU)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn


@pytest.mark.parametrize("cast", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("made", [torch.bfloat16, torch.float32])
def test_a_module_that_was_cast(made, cast):
    """Weights and scale in the type of the cast; the call takes the scale in FP32."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, r, g, dh, dz = (torch.randn(37, 256, generator=gen, device="cuda").bfloat16() for _ in range(5))
    mod = gn.BlockRMSNorm(256, alpha=0.5, dtype=made, device="cuda").to(cast)
    assert {p.dtype for p in mod.parameters()} == {cast}
    torch.autograd.backward(mod(a, r, g), [dh, dz])
    w, alpha = torch.ones(256, dtype=cast, device="cuda"), torch.full((1,), 0.5, device="cuda")
    h, z, r1, r2 = gn.gnorm_block_fwd(a, r, w, w, g=g, alpha=alpha)
    _, _, _, dw1, dw2, dalpha = gn.gnorm_block_bwd(dh, dz, a, r, w, w, r1, r2, g=g, alpha=alpha,
                                                   dw_fp32=cast == torch.float32)
    assert torch.equal(mod.weight_post.grad, dw1) and torch.equal(mod.weight_pre.grad, dw2)
    assert torch.equal(mod.alpha.grad, dalpha.to(cast))
    out = mod(a, r, g)
    assert torch.equal(out[0], h) and torch.equal(out[1], z)
