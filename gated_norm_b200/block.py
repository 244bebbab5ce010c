"""Block norm: the norm after a block, its gate, the residual scale and the norm before the
next block in one pass (``gnorm_block_fwd`` / ``gnorm_block_bwd`` of include/gnorm.h), and its
torch.autograd form.

Argument marshalling only; every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import GnormBlockBwdDesc, GnormBlockFwdDesc, lib
from .gnorm import _check, _device_buffer, _on, _ptr, _same, _stream, _vec

__all__ = ["gnorm_block_fwd", "gnorm_block_bwd", "gnorm_block_bwd_workspace_bytes",
           "block_rmsnorm", "BlockRMSNormFunction", "BlockRMSNorm"]

_RES = (torch.bfloat16, torch.float32)
_BF16 = (torch.bfloat16,)
_FP32 = (torch.float32,)


def _rows(t: torch.Tensor, name: str, dtypes, like=None):
    """Row stride of rows of the last dimension: contiguous of any rank, or a 2-D view with unit
    column stride."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None:
        if t.shape != like.shape or t.device != like.device:
            _same(like, t, "a", name)
    elif t.dim() < 1:
        raise ValueError(f"{name} must have a last dimension N")
    if t.is_contiguous():
        return t.shape[-1]
    if t.dim() == 2 and t.stride(1) == 1:
        return t.stride(0) if t.shape[0] > 1 else t.shape[1]
    raise ValueError(f"{name}: rows need unit column stride (2-D row-strided views or "
                     "contiguous tensors)")


def _common(d, a, r, g, w1, w2, alpha):
    """Checks the inputs that both calls share and puts them into the descriptor."""
    d.lda = _rows(a, "a", _BF16)
    N = a.shape[-1]
    M = a.numel() // N if N else 0
    d.ldr = _rows(r, "r", _RES, a)
    if g is not None:
        d.ldg = _rows(g, "g", _BF16, a)
        d.g = _ptr(g)
    dev = a.device
    _vec(w1, N, _RES, "w1", dev)
    _vec(w2, N, (w1.dtype,), "w2", dev)
    if alpha is not None:
        _vec(alpha, 1, _FP32, "alpha", dev)
        d.alpha = alpha.data_ptr()
    d.a, d.r, d.w1, d.w2 = _ptr(a), _ptr(r), _ptr(w1), _ptr(w2)
    d.w_fp32, d.res_fp32 = w1.dtype == torch.float32, r.dtype == torch.float32
    d.M, d.N = M, N
    return M, N, dev


def gnorm_block_fwd(a, r, w1, w2, eps: float = 1e-6, *, g=None, alpha=None, eps2=None, h=None,
                    z=None, rstd1=None, rstd2=None, stream=None):
    """Forward: returns (h, z, rstd1, rstd2).

    h = r + alpha * silu(g) * rmsnorm(a) * w1 and z = rmsnorm(h) * w2.  a, g: BF16 rows; r:
    BF16 or FP32 rows (h has its type); w1, w2: both BF16 or both FP32 [N]; alpha: FP32 [1] on
    the device, None = 1; g None = no gate; eps2: the second norm's eps (None = eps)."""
    d = GnormBlockFwdDesc()
    M, _, dev = _common(d, a, r, g, w1, w2, alpha)
    if h is None:
        h = torch.empty(a.shape, dtype=r.dtype, device=dev)
    if z is None:
        z = torch.empty(a.shape, dtype=torch.bfloat16, device=dev)
    if rstd1 is None and rstd2 is None:
        rstd1, rstd2 = torch.empty((2, M), dtype=torch.float32, device=dev).unbind()
    else:
        if rstd1 is None:
            rstd1 = torch.empty(M, dtype=torch.float32, device=dev)
        if rstd2 is None:
            rstd2 = torch.empty(M, dtype=torch.float32, device=dev)
        _vec(rstd1, M, _FP32, "rstd1", dev)
        _vec(rstd2, M, _FP32, "rstd2", dev)
    d.eps1, d.eps2 = eps, eps if eps2 is None else eps2
    d.h, d.ldh, d.z, d.ldz = _ptr(h), _rows(h, "h", (r.dtype,), a), _ptr(z), _rows(z, "z", _BF16, a)
    d.rstd1, d.rstd2 = _ptr(rstd1), _ptr(rstd2)
    with _on(dev):
        st = lib.gnorm_block_fwd(ctypes.byref(d), _stream(stream, dev))
    _check(st, "gnorm_block_fwd")
    return h, z, rstd1, rstd2


def gnorm_block_bwd_workspace_bytes(M: int, N: int) -> int:
    return int(lib.gnorm_block_bwd_workspace_bytes(int(M), int(N)))


def gnorm_block_bwd(dh, dz, a, r, w1, w2, rstd1, rstd2, *, g=None, alpha=None, da=None, dr=None,
                    dg=None, dw1=None, dw2=None, dalpha=None, dw_fp32: bool = False,
                    workspace_buf=None, stream=None):
    """Backward: returns (da, dr, dg, dw1, dw2, dalpha); dg is None without a gate, dalpha
    without an alpha.

    dh: gradient of h through the residual (r's type; None = zero); dz: BF16 gradient of z;
    rstd1, rstd2 as the forward wrote them.  dw1 and dw2 are FP32 if dw_fp32 else BF16."""
    d = GnormBlockBwdDesc()
    M, N, dev = _common(d, a, r, g, w1, w2, alpha)
    if dh is not None:
        d.dh, d.lddh = _ptr(dh), _rows(dh, "dh", (r.dtype,), a)
    d.dz, d.lddz = _ptr(dz), _rows(dz, "dz", _BF16, a)
    _vec(rstd1, M, _FP32, "rstd1", dev)
    _vec(rstd2, M, _FP32, "rstd2", dev)
    d.rstd1, d.rstd2 = _ptr(rstd1), _ptr(rstd2)
    if da is None:
        da = torch.empty(a.shape, dtype=torch.bfloat16, device=dev)
    if dr is None:
        dr = torch.empty(a.shape, dtype=r.dtype, device=dev)
    d.da, d.ldda = _ptr(da), _rows(da, "da", _BF16, a)
    d.dr, d.lddr = _ptr(dr), _rows(dr, "dr", (r.dtype,), a)
    if g is not None:
        if dg is None:
            dg = torch.empty(a.shape, dtype=torch.bfloat16, device=dev)
        d.dg, d.lddg = _ptr(dg), _rows(dg, "dg", _BF16, a)
    elif dg is not None:
        raise ValueError("dg without a gate")
    wt = torch.float32 if dw_fp32 else torch.bfloat16
    dw1 = torch.empty(N, dtype=wt, device=dev) if dw1 is None else dw1
    dw2 = torch.empty(N, dtype=wt, device=dev) if dw2 is None else dw2
    _vec(dw1, N, (wt,), "dw1", dev)
    _vec(dw2, N, (wt,), "dw2", dev)
    d.dw1, d.dw2, d.dw_fp32 = _ptr(dw1), _ptr(dw2), bool(dw_fp32)
    if alpha is not None:
        dalpha = torch.empty_like(alpha) if dalpha is None else dalpha
        _vec(dalpha, 1, _FP32, "dalpha", dev)
        d.dalpha = dalpha.data_ptr()
    elif dalpha is not None:
        raise ValueError("dalpha without an alpha")
    with _on(dev):
        if workspace_buf is None:
            # from torch's allocator for every call: ordered on the stream that uses it, and
            # owned by the graph when the call is captured
            need = gnorm_block_bwd_workspace_bytes(M, N)
            if stream is None:
                workspace_buf = torch.empty(need, dtype=torch.uint8, device=dev)
            else:
                with torch.cuda.stream(stream):
                    workspace_buf = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _device_buffer(workspace_buf, "workspace_buf", dev)
        d.workspace = _ptr(workspace_buf)
        d.workspace_bytes = workspace_buf.numel() * workspace_buf.element_size()
        st = lib.gnorm_block_bwd(ctypes.byref(d), _stream(stream, dev))
    _check(st, "gnorm_block_bwd")
    return da, dr, dg, dw1, dw2, dalpha


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
        dh = None if dh is None else dh.contiguous()
        dz = torch.zeros(a.shape, dtype=a.dtype, device=a.device) if dz is None \
            else dz.contiguous()
        da, dr, dg, dw1, dw2, dalpha = gnorm_block_bwd(
            dh, dz, a, r, w1, w2, rstd1, rstd2, g=g, alpha=alpha,
            dw_fp32=w1.dtype == torch.float32)
        return da, dr, dg, dw1, dw2, dalpha, None, None


def block_rmsnorm(a, r, w1, w2, eps: float = 1e-6, *, g=None, alpha=None, eps2=None):
    """(h, z) of gnorm_block_fwd, differentiable in a, r, g, w1, w2 and alpha."""
    return BlockRMSNormFunction.apply(a, r, g, w1, w2, alpha, eps, eps if eps2 is None else eps2)


class BlockRMSNorm(torch.nn.Module):
    """Module form: the two learnable weights and the learnable residual scale (FP32 [1])."""

    def __init__(self, n: int, eps: float = 1e-6, *, alpha: float = 1.0, dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        self.weight_post = torch.nn.Parameter(torch.ones(n, dtype=dtype, device=device))
        self.weight_pre = torch.nn.Parameter(torch.ones(n, dtype=dtype, device=device))
        self.alpha = torch.nn.Parameter(torch.full((1,), float(alpha), device=device))
        self.eps = eps

    def forward(self, a, r, g=None):
        return block_rmsnorm(a, r, self.weight_post, self.weight_pre, self.eps, g=g,
                             alpha=self.alpha)
