"""The gated delta rule (``gnorm_delta_fwd`` / ``gnorm_delta_bwd`` / ``gnorm_delta_step`` of
include/gnorm.h), its torch.autograd form, and the rule with the gated norm behind it.

The arguments are checked in the module _marshal; every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import torch

from . import _marshal
from ._lib import lib
from .autograd import _grad, gated_rmsnorm
from .gnorm import _check, _handle

__all__ = ["gnorm_delta_fwd", "gnorm_delta_bwd", "gnorm_delta_step",
           "gnorm_delta_workspace_bytes", "GatedDeltaRuleFunction", "gated_delta_rule",
           "GatedDeltaNorm"]

def gnorm_delta_workspace_bytes(T: int, B: int, Hv: int, K: int, V: int,
                                backward: bool = False) -> int:
    return int(lib.gnorm_delta_workspace_bytes(int(T), int(B), int(Hv), int(K), int(V),
                                               int(bool(backward))))


def gnorm_delta_fwd(q, k, v, g, beta, *, scale=None, cu_seqlens=None, initial_state=None,
                    output_final_state: bool = False, o=None, final_state=None,
                    workspace_buf=None, stream=None):
    """Forward over whole sequences: returns (o, final_state); final_state is None unless asked
    for.

    q, k: BF16 [T, Hk, K]; v: BF16 [T, Hv, V]; g: FP32 [T, Hv], the log of the decay; beta:
    BF16 or FP32 [T, Hv]; scale: None = K**-0.5.  cu_seqlens (int32 [B + 1], on the device)
    packs B sequences into the T tokens; without it [T, ...] is one sequence and [B, L, ...]
    are B.  States are FP32 [B, Hv, K, V].  Rows of o behind the last sequence are zero if this
    call allocates o, and left as they are in an o that is passed in."""
    st, o, final_state = _marshal.delta_fwd(q, k, v, g, beta, scale, cu_seqlens, initial_state,
                                            output_final_state, o, final_state, workspace_buf,
                                            _handle(stream))
    _check(st, "gnorm_delta_fwd")
    return o, final_state


def gnorm_delta_bwd(do, q, k, v, g, beta, *, scale=None, cu_seqlens=None, initial_state=None,
                    dfinal_state=None, dq=None, dk=None, dv=None, dg=None, dbeta=None,
                    dinitial_state=None, workspace_buf=None, stream=None):
    """Backward: returns (dq, dk, dv, dg, dbeta, dinitial_state) from do, the gradient of o, and
    dfinal_state, the final state's (None = zero), with the forward's inputs.

    dq, dk and dv are BF16, dg is FP32, dbeta has beta's type; dinitial_state is None without
    an initial state.  Rows behind the last sequence are zero in gradients that this call
    allocates and left as they are in ones that are passed in; with cu_seqlens pass all of dq, dk,
    dv, dg and dbeta, or none."""
    st, *out = _marshal.delta_bwd(do, q, k, v, g, beta, scale, cu_seqlens, initial_state,
                                  dfinal_state, dq, dk, dv, dg, dbeta, dinitial_state,
                                  workspace_buf, _handle(stream))
    _check(st, "gnorm_delta_bwd")
    return tuple(out)


def gnorm_delta_step(q, k, v, g, beta, state, *, slots=None, scale=None, o=None, stream=None):
    """One token of each of B sequences: returns o and updates ``state`` in place.

    q, k: BF16 [B, Hk, K]; v: BF16 [B, Hv, V]; g: FP32 [B, Hv]; beta: BF16 or FP32 [B, Hv];
    state: FP32 [pool, Hv, K, V], slots any distance apart; slots: int32 [B] on the device, row
    b's place in the pool (None: b).  A slot outside the pool marks a padded row: its o is
    zero and no state is touched.  Rows that share a slot are tokens of one sequence, in row
    order."""
    st, o = _marshal.delta_step(q, k, v, g, beta, state, slots, scale, o, _handle(stream))
    _check(st, "gnorm_delta_step")
    return o


class GatedDeltaRuleFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, cu_seqlens, scale):
        o, final = gnorm_delta_fwd(q, k, v, g, beta, scale=scale, cu_seqlens=cu_seqlens,
                                   initial_state=initial_state, output_final_state=True)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dfinal):
        q, k, v, g, beta, initial_state, cu_seqlens = ctx.saved_tensors
        do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None \
            else _grad(do)
        dfinal = None if dfinal is None else _grad(dfinal)
        dq, dk, dv, dg, dbeta, ds = gnorm_delta_bwd(
            do, q, k, v, g, beta, scale=ctx.scale, cu_seqlens=cu_seqlens,
            initial_state=initial_state, dfinal_state=dfinal)
        return dq, dk, dv, dg, dbeta, ds, None, None


def gated_delta_rule(q, k, v, g, beta, *, scale=None, cu_seqlens=None, initial_state=None):
    """(o, final_state) of gnorm_delta_fwd, differentiable in q, k, v, g, beta and
    initial_state."""
    return GatedDeltaRuleFunction.apply(q, k, v, g, beta, initial_state, cu_seqlens, scale)


class GatedDeltaNorm(torch.nn.Module):
    """The core of a linear-attention layer: the gated delta rule, then the gated norm of every
    head's output (a learnable weight of size V, shared by the heads)."""

    def __init__(self, head_v_dim: int, eps: float = 1e-6, *, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(head_v_dim, dtype=dtype, device=device))
        self.eps = eps

    def forward(self, q, k, v, g, beta, gate, *, scale=None, cu_seqlens=None, initial_state=None):
        """(y, final_state) over whole sequences; gate: BF16, v's shape (a slice of a wider
        projection is copied: the norm's rows are all one distance apart).  The norm takes every
        row, so gate has to be finite behind the last sequence too."""
        o, final = gated_delta_rule(q, k, v, g, beta, scale=scale, cu_seqlens=cu_seqlens,
                                    initial_state=initial_state)
        return gated_rmsnorm(o, gate.contiguous(), self.weight, self.eps), final

    def step(self, q, k, v, g, beta, gate, state, *, slots=None, scale=None):
        """y for one token of each sequence; ``state`` is updated in place (no gradients)."""
        with torch.no_grad():
            o = gnorm_delta_step(q, k, v, g, beta, state, slots=slots, scale=scale)
            return gated_rmsnorm(o, gate.contiguous(), self.weight, self.eps)
