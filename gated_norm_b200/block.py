"""Block norm: the norm after a block, its gate, the residual scale and the norm before the
next block in one pass (``gnorm_block_fwd`` / ``gnorm_block_bwd`` of include/gnorm.h), and its
torch.autograd form.

The arguments are checked in the module _marshal; every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import torch

from . import _marshal
from ._lib import lib
from .autograd import _grad
from .gnorm import _check, _handle

__all__ = ["gnorm_block_fwd", "gnorm_block_bwd", "gnorm_block_bwd_workspace_bytes",
           "block_rmsnorm", "BlockRMSNormFunction", "BlockRMSNorm"]

def gnorm_block_fwd(a, r, w1, w2, eps: float = 1e-6, *, g=None, alpha=None, eps2=None, h=None,
                    z=None, rstd1=None, rstd2=None, stream=None):
    """Forward: returns (h, z, rstd1, rstd2).

    h = r + alpha * silu(g) * rmsnorm(a) * w1 and z = rmsnorm(h) * w2.  a, g: BF16 rows; r:
    BF16 or FP32 rows (h has its type); w1, w2: both BF16 or both FP32 [N]; alpha: FP32 [1] on
    the device, None = 1; g None = no gate; eps2: the second norm's eps (None = eps)."""
    st, *out = _marshal.block_fwd(a, r, w1, w2, eps, eps if eps2 is None else eps2, g, alpha, h,
                                  z, rstd1, rstd2, _handle(stream))
    _check(st, "gnorm_block_fwd")
    return tuple(out)


def gnorm_block_bwd_workspace_bytes(M: int, N: int) -> int:
    return int(lib.gnorm_block_bwd_workspace_bytes(int(M), int(N)))


def gnorm_block_bwd(dh, dz, a, r, w1, w2, rstd1, rstd2, *, g=None, alpha=None, da=None, dr=None,
                    dg=None, dw1=None, dw2=None, dalpha=None, dw_fp32: bool = False,
                    workspace_buf=None, stream=None):
    """Backward: returns (da, dr, dg, dw1, dw2, dalpha); dg is None without a gate, dalpha
    without an alpha.

    dh: gradient of h through the residual (r's type; None = zero); dz: BF16 gradient of z;
    rstd1, rstd2 as the forward wrote them.  dw1 and dw2 are FP32 if dw_fp32 else BF16."""
    st, *out = _marshal.block_bwd(dh, dz, a, r, w1, w2, rstd1, rstd2, g, alpha, da, dr, dg, dw1,
                                  dw2, dalpha, dw_fp32, workspace_buf, _handle(stream))
    _check(st, "gnorm_block_bwd")
    return tuple(out)


class BlockRMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, r, g, w1, w2, alpha, eps: float, eps2: float):
        h, z, rstd1, rstd2 = gnorm_block_fwd(a, r, w1, w2, eps, g=g, alpha=alpha, eps2=eps2)
        ctx.save_for_backward(a, r, g, w1, w2, alpha, rstd1, rstd2)
        ctx.set_materialize_grads(False)
        return h, z

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dz):
        a, r, g, w1, w2, alpha, rstd1, rstd2 = ctx.saved_tensors
        dh = None if dh is None else _grad(dh)
        dz = torch.zeros(a.shape, dtype=a.dtype, device=a.device) if dz is None \
            else _grad(dz)
        da, dr, dg, dw1, dw2, dalpha = gnorm_block_bwd(
            dh, dz, a, r, w1, w2, rstd1, rstd2, g=g, alpha=alpha,
            dw_fp32=w1.dtype == torch.float32)
        return da, dr, dg, dw1, dw2, dalpha, None, None


def block_rmsnorm(a, r, w1, w2, eps: float = 1e-6, *, g=None, alpha=None, eps2=None):
    """(h, z) of gnorm_block_fwd, differentiable in a, r, g, w1, w2 and alpha."""
    return BlockRMSNormFunction.apply(a, r, g, w1, w2, alpha, eps, eps if eps2 is None else eps2)


class BlockRMSNorm(torch.nn.Module):
    """Module form: the two learnable weights and the learnable residual scale ([1], FP32 in the
    call whatever type the module has been cast to)."""

    def __init__(self, n: int, eps: float = 1e-6, *, alpha: float = 1.0, dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        self.weight_post = torch.nn.Parameter(torch.ones(n, dtype=dtype, device=device))
        self.weight_pre = torch.nn.Parameter(torch.ones(n, dtype=dtype, device=device))
        self.alpha = torch.nn.Parameter(torch.full((1,), float(alpha), device=device))
        self.eps = eps

    def forward(self, a, r, g=None):
        return block_rmsnorm(a, r, self.weight_post, self.weight_pre, self.eps, g=g,
                             alpha=self.alpha.float())
