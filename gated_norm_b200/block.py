"""Block norm: the norm after a block, its gate, the residual scale and the norm before the
next block in one pass (``gnorm_block_fwd`` / ``gnorm_block_bwd`` of include/gnorm.h), and its
torch.autograd form.

Argument marshalling only; every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import GnormBlockBwdDesc, GnormBlockFwdDesc, lib
from .gnorm import _check, _device_buffer, _ptr, _same, _stream, _vec

__all__ = ["gnorm_block_fwd", "gnorm_block_bwd", "gnorm_block_bwd_workspace_bytes",
           "block_rmsnorm", "BlockRMSNormFunction", "BlockRMSNorm"]

_RES = (torch.bfloat16, torch.float32)


def _rows(t: torch.Tensor, name: str, dtypes):
    """(M, N, row stride): contiguous of any rank, or a 2-D view with unit column stride."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() < 1:
        raise ValueError(f"{name} must have a last dimension N")
    N = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // N if N else 0), N, N
    if t.dim() == 2 and t.stride(1) == 1:
        return t.shape[0], N, (t.stride(0) if t.shape[0] > 1 else N)
    raise ValueError(f"{name}: rows need unit column stride (2-D row-strided views or "
                     "contiguous tensors)")


def _common(a, r, g, w1, w2, alpha):
    M, N, lda = _rows(a, "a", (torch.bfloat16,))
    _same(a, r, "a", "r")
    _, _, ldr = _rows(r, "r", _RES)
    ldg = 0
    if g is not None:
        _same(a, g, "a", "g")
        _, _, ldg = _rows(g, "g", (torch.bfloat16,))
    _vec(w1, N, _RES, "w1", a.device)
    _vec(w2, N, (w1.dtype,), "w2", a.device)
    if alpha is not None:
        _vec(alpha, 1, (torch.float32,), "alpha", a.device)
    return M, N, dict(a=_ptr(a), lda=lda, r=_ptr(r), ldr=ldr, g=_ptr(g), ldg=ldg, w1=_ptr(w1),
                      w2=_ptr(w2), w_fp32=int(w1.dtype == torch.float32),
                      res_fp32=int(r.dtype == torch.float32), alpha=_ptr(alpha), M=M, N=N)


def _out(t, like, dtype, name):
    if t is None:
        return torch.empty(like.shape, dtype=dtype, device=like.device)
    _same(like, t, "a", name)
    return t


def gnorm_block_fwd(a, r, w1, w2, eps: float = 1e-6, *, g=None, alpha=None, eps2=None, h=None,
                    z=None, rstd1=None, rstd2=None, stream=None):
    """Forward: returns (h, z, rstd1, rstd2).

    h = r + alpha * silu(g) * rmsnorm(a) * w1 and z = rmsnorm(h) * w2.  a, g: BF16 rows; r:
    BF16 or FP32 rows (h has its type); w1, w2: both BF16 or both FP32 [N]; alpha: FP32 [1] on
    the device, None = 1; g None = no gate; eps2: the second norm's eps (None = eps)."""
    M, N, c = _common(a, r, g, w1, w2, alpha)
    h = _out(h, a, r.dtype, "h")
    z = _out(z, a, torch.bfloat16, "z")
    _, _, ldh = _rows(h, "h", (r.dtype,))
    _, _, ldz = _rows(z, "z", (torch.bfloat16,))
    if rstd1 is None or rstd2 is None:
        both = torch.empty((2, M), dtype=torch.float32, device=a.device)
        rstd1 = both[0] if rstd1 is None else rstd1
        rstd2 = both[1] if rstd2 is None else rstd2
    for t, n in ((rstd1, "rstd1"), (rstd2, "rstd2")):
        _vec(t, M, (torch.float32,), n, a.device)
    d = GnormBlockFwdDesc(eps1=float(eps), eps2=float(eps if eps2 is None else eps2), h=_ptr(h),
                          ldh=ldh, z=_ptr(z), ldz=ldz, rstd1=_ptr(rstd1), rstd2=_ptr(rstd2), **c)
    with torch.cuda.device(a.device):
        st = lib.gnorm_block_fwd(ctypes.byref(d), _stream(stream, a.device))
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
    M, N, c = _common(a, r, g, w1, w2, alpha)
    dev = a.device
    lddh = 0
    if dh is not None:
        _same(a, dh, "a", "dh")
        _, _, lddh = _rows(dh, "dh", (r.dtype,))
    _same(a, dz, "a", "dz")
    _, _, lddz = _rows(dz, "dz", (torch.bfloat16,))
    for t, n in ((rstd1, "rstd1"), (rstd2, "rstd2")):
        _vec(t, M, (torch.float32,), n, dev)
    da = _out(da, a, torch.bfloat16, "da")
    dr = _out(dr, a, r.dtype, "dr")
    _, _, ldda = _rows(da, "da", (torch.bfloat16,))
    _, _, lddr = _rows(dr, "dr", (r.dtype,))
    lddg = 0
    if g is not None:
        dg = _out(dg, a, torch.bfloat16, "dg")
        _, _, lddg = _rows(dg, "dg", (torch.bfloat16,))
    elif dg is not None:
        raise ValueError("dg without a gate")
    wt = torch.float32 if dw_fp32 else torch.bfloat16
    dw1 = torch.empty(N, dtype=wt, device=dev) if dw1 is None else dw1
    dw2 = torch.empty(N, dtype=wt, device=dev) if dw2 is None else dw2
    for t, n in ((dw1, "dw1"), (dw2, "dw2")):
        _vec(t, N, (wt,), n, dev)
    if alpha is not None:
        dalpha = torch.empty_like(alpha) if dalpha is None else dalpha
        _vec(dalpha, 1, (torch.float32,), "dalpha", dev)
    elif dalpha is not None:
        raise ValueError("dalpha without an alpha")
    with torch.cuda.device(dev):
        if workspace_buf is None:
            # from torch's allocator for every call: ordered on the stream that uses it, and
            # owned by the graph when the call is captured
            with torch.cuda.stream(stream or torch.cuda.current_stream(dev)):
                workspace_buf = torch.empty(gnorm_block_bwd_workspace_bytes(M, N),
                                            dtype=torch.uint8, device=dev)
        else:
            _device_buffer(workspace_buf, "workspace_buf", dev)
        d = GnormBlockBwdDesc(
            dh=_ptr(dh), lddh=lddh, dz=_ptr(dz), lddz=lddz, rstd1=_ptr(rstd1), rstd2=_ptr(rstd2),
            da=_ptr(da), ldda=ldda, dr=_ptr(dr), lddr=lddr, dg=_ptr(dg), lddg=lddg,
            dw1=_ptr(dw1), dw2=_ptr(dw2), dw_fp32=int(bool(dw_fp32)), dalpha=_ptr(dalpha),
            workspace=_ptr(workspace_buf),
            workspace_bytes=workspace_buf.numel() * workspace_buf.element_size(), **c)
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
