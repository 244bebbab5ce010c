"""The gated delta rule (``gnorm_delta_fwd`` / ``gnorm_delta_bwd`` / ``gnorm_delta_step`` of
include/gnorm.h), its torch.autograd form, and the rule with the gated norm behind it.

Argument marshalling only; every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import GnormDeltaBwdDesc, GnormDeltaFwdDesc, GnormDeltaIn, GnormDeltaStepDesc, lib
from .autograd import gated_rmsnorm
from .gnorm import _check, _device_buffer, _on, _ptr, _stream

__all__ = ["gnorm_delta_fwd", "gnorm_delta_bwd", "gnorm_delta_step",
           "gnorm_delta_workspace_bytes", "GatedDeltaRuleFunction", "gated_delta_rule",
           "GatedDeltaNorm"]

_BF16 = (torch.bfloat16,)
_FP32 = (torch.float32,)
_BETA = _BF16 + _FP32


def _tokens(t: torch.Tensor, name: str, tail, dtypes, lead, device):
    """Token stride of a [*lead, *tail] CUDA tensor ([T, ...] or [B, L, ...]) whose heads are
    packed within a token (tokens may be any distance apart, e.g. a slice of a wider
    projection)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    if t.shape != lead + tail:
        raise ValueError(f"{name} must be {lead + tail}, got {tuple(t.shape)}")
    width = tail[0] * tail[1] if len(tail) == 2 else tail[0]
    if t.is_contiguous() or t.numel() == 0:
        return width
    st, n = t.stride(), len(lead)
    want = 1
    for size, step in zip(tail[::-1], st[:n - 1:-1]):
        if size > 1 and step != want:
            raise ValueError(f"{name}: the heads of a token must be packed, strides {st}")
        want *= size
    if n == 1:
        return st[0] if lead[0] > 1 else width
    ld = st[1] if lead[1] > 1 else (st[0] if lead[0] > 1 else width)
    if lead[0] > 1 and st[0] != ld * lead[1]:
        raise ValueError(f"{name}: tokens must be evenly spaced over the batch, strides {st}")
    return ld


def _state(t, name: str, shape, device):
    if t is None:
        return
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.device != device or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on {device}, got "
                         f"{tuple(t.shape)} on {t.device}")


def _inputs(d, q, k, v, g, beta, scale, cu_seqlens, initial_state):
    """Checks the inputs that both calls share and puts them into the descriptor; returns the
    leading and the state shape."""
    if q.dim() not in (3, 4) or v.dim() != q.dim():
        raise ValueError("q, k and v must be [T, heads, dim] or [B, L, heads, dim]")
    lead, qk, vv = q.shape[:-2], q.shape[-2:], v.shape[-2:]
    (Hk, K), (Hv, V) = qk, vv
    dev = q.device
    d.ldq, d.q = _tokens(q, "q", qk, _BF16, lead, dev), _ptr(q)
    d.ldk, d.k = _tokens(k, "k", qk, _BF16, lead, dev), _ptr(k)
    d.ldv, d.v = _tokens(v, "v", vv, _BF16, lead, dev), _ptr(v)
    d.ldg, d.g = _tokens(g, "g", (Hv,), _FP32, lead, dev), _ptr(g)
    d.ldbeta, d.beta = _tokens(beta, "beta", (Hv,), _BETA, lead, dev), _ptr(beta)
    d.beta_fp32 = beta.dtype == torch.float32
    d.Hk, d.Hv, d.K, d.V = Hk, Hv, K, V
    d.scale = K ** -0.5 if scale is None else scale
    if cu_seqlens is not None:
        if len(lead) != 1:
            raise ValueError("cu_seqlens goes with [T, heads, dim] tensors")
        if cu_seqlens.dtype != torch.int32:
            raise TypeError(f"cu_seqlens must be int32, got {cu_seqlens.dtype}")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous() or \
                cu_seqlens.device != dev:
            raise ValueError(f"cu_seqlens must be a contiguous [B + 1] tensor on {dev}")
        d.cu_seqlens, d.B, d.T = _ptr(cu_seqlens), cu_seqlens.numel() - 1, lead[0]
    elif len(lead) == 2:
        d.B, d.T = lead[0], lead[0] * lead[1]
    else:
        d.B, d.T = 1, lead[0]
    shape = (d.B, Hv, K, V)
    _state(initial_state, "initial_state", shape, dev)
    d.initial_state = _ptr(initial_state)
    return lead, shape


def gnorm_delta_workspace_bytes(T: int, B: int, Hv: int, K: int, V: int,
                                backward: bool = False) -> int:
    return int(lib.gnorm_delta_workspace_bytes(int(T), int(B), int(Hv), int(K), int(V),
                                               int(bool(backward))))


def _workspace(buf, d, backward, device, stream):
    if buf is None:
        # from torch's allocator for every call: ordered on the stream that uses it, and
        # owned by the graph when the call is captured
        need = gnorm_delta_workspace_bytes(d.T, d.B, d.Hv, d.K, d.V, backward)
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=device)
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=device)
    _device_buffer(buf, "workspace_buf", device)
    return buf


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
    f = GnormDeltaFwdDesc()
    d = getattr(f, "in")  # shares f's memory
    lead, shape = _inputs(d, q, k, v, g, beta, scale, cu_seqlens, initial_state)
    dev = q.device
    own = o is None
    if own:
        o = torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
    f.ldo, f.o = _tokens(o, "o", v.shape[-2:], _BF16, lead, dev), _ptr(o)
    if final_state is None and output_final_state:
        final_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(final_state, "final_state", shape, dev)
    f.final_state = _ptr(final_state)
    f.zero_tail = own and cu_seqlens is not None
    with _on(dev):
        ws = _workspace(workspace_buf, d, False, dev, stream)
        f.workspace, f.workspace_bytes = _ptr(ws), ws.numel() * ws.element_size()
        st = lib.gnorm_delta_fwd(ctypes.byref(f), _stream(stream, dev))
    _check(st, "gnorm_delta_fwd")
    return o, final_state


def gnorm_delta_bwd(do, q, k, v, g, beta, *, scale=None, cu_seqlens=None, initial_state=None,
                    dfinal_state=None, dq=None, dk=None, dv=None, dg=None, dbeta=None,
                    dinitial_state=None, workspace_buf=None, stream=None):
    """Backward: returns (dq, dk, dv, dg, dbeta, dinitial_state) from do, the gradient of o, and
    dfinal_state, the final state's (None = zero), with the forward's inputs.

    dq, dk and dv are BF16, dg is FP32, dbeta has beta's type; dinitial_state is None without
    an initial state.  Rows behind the last sequence are zero in gradients that this call
    allocates; if any is passed in, they are left as they are in all of them."""
    b = GnormDeltaBwdDesc()
    d = getattr(b, "in")  # shares b's memory
    lead, shape = _inputs(d, q, k, v, g, beta, scale, cu_seqlens, initial_state)
    dev = q.device
    qk, vv, gb = q.shape[-2:], v.shape[-2:], g.shape[-1:]
    b.lddo, b.d_o = _tokens(do, "do", vv, _BF16, lead, dev), _ptr(do)
    _state(dfinal_state, "dfinal_state", shape, dev)
    given = [t is not None for t in (dq, dk, dv, dg, dbeta)]
    if cu_seqlens is not None and any(given) and not all(given):
        raise ValueError("with cu_seqlens pass all of dq, dk, dv, dg and dbeta, or none")
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev) if dq is None else dq
    dk = torch.empty(k.shape, dtype=k.dtype, device=dev) if dk is None else dk
    dv = torch.empty(v.shape, dtype=v.dtype, device=dev) if dv is None else dv
    dg = torch.empty(g.shape, dtype=g.dtype, device=dev) if dg is None else dg
    dbeta = torch.empty(beta.shape, dtype=beta.dtype, device=dev) if dbeta is None else dbeta
    b.lddq, b.dq = _tokens(dq, "dq", qk, _BF16, lead, dev), _ptr(dq)
    b.lddk, b.dk = _tokens(dk, "dk", qk, _BF16, lead, dev), _ptr(dk)
    b.lddv, b.dv = _tokens(dv, "dv", vv, _BF16, lead, dev), _ptr(dv)
    b.lddg, b.dg = _tokens(dg, "dg", gb, _FP32, lead, dev), _ptr(dg)
    b.lddbeta, b.dbeta = _tokens(dbeta, "dbeta", gb, (beta.dtype,), lead, dev), _ptr(dbeta)
    if dinitial_state is None and initial_state is not None:
        dinitial_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(dinitial_state, "dinitial_state", shape, dev)
    b.dfinal_state, b.dinitial_state = _ptr(dfinal_state), _ptr(dinitial_state)
    b.zero_tail = cu_seqlens is not None and not any(given)
    with _on(dev):
        ws = _workspace(workspace_buf, d, True, dev, stream)
        b.workspace, b.workspace_bytes = _ptr(ws), ws.numel() * ws.element_size()
        st = lib.gnorm_delta_bwd(ctypes.byref(b), _stream(stream, dev))
    _check(st, "gnorm_delta_bwd")
    return dq, dk, dv, dg, dbeta, dinitial_state


def gnorm_delta_step(q, k, v, g, beta, state, *, slots=None, scale=None, o=None, stream=None):
    """One token of each of B sequences: returns o and updates ``state`` in place.

    q, k: BF16 [B, Hk, K]; v: BF16 [B, Hv, V]; g: FP32 [B, Hv]; beta: BF16 or FP32 [B, Hv];
    state: FP32 [pool, Hv, K, V], slots any distance apart; slots: int32 [B] on the device, row
    b's place in the pool (None: b).  A slot outside the pool marks a padded row: its o is
    zero and no state is touched.  Rows that share a slot are tokens of one sequence, in row
    order."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [B, heads, dim]")
    lead, qk, vv = q.shape[:1], q.shape[1:], v.shape[1:]
    (Hk, K), (Hv, V) = qk, vv
    dev = q.device
    if state.dtype != torch.float32:
        raise TypeError(f"state must be float32, got {state.dtype}")
    if state.dim() != 4 or state.shape[1:] != (Hv, K, V) or state.device != dev or \
            not (state.is_contiguous() or state[:1].is_contiguous()):
        raise ValueError(f"state must be [pool, {Hv}, {K}, {V}] on {dev} with packed slots, got "
                         f"{tuple(state.shape)} on {state.device}")
    if slots is not None:
        if slots.dtype != torch.int32:
            raise TypeError(f"slots must be int32, got {slots.dtype}")
        if slots.shape != lead or not slots.is_contiguous() or slots.device != dev:
            raise ValueError(f"slots must be a contiguous [{lead[0]}] tensor on {dev}")
    if o is None:
        o = torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
    d = GnormDeltaStepDesc()
    d.ldq, d.q = _tokens(q, "q", qk, _BF16, lead, dev), _ptr(q)
    d.ldk, d.k = _tokens(k, "k", qk, _BF16, lead, dev), _ptr(k)
    d.ldv, d.v = _tokens(v, "v", vv, _BF16, lead, dev), _ptr(v)
    d.ldg, d.g = _tokens(g, "g", (Hv,), _FP32, lead, dev), _ptr(g)
    d.ldbeta, d.beta = _tokens(beta, "beta", (Hv,), _BETA, lead, dev), _ptr(beta)
    d.beta_fp32 = beta.dtype == torch.float32
    d.B, d.Hk, d.Hv, d.K, d.V = lead[0], Hk, Hv, K, V
    d.scale = K ** -0.5 if scale is None else scale
    d.state, d.pool = _ptr(state), state.shape[0]
    d.ldstate = state.stride(0) if state.shape[0] > 1 else Hv * K * V
    d.slots = _ptr(slots)
    d.ldo, d.o = _tokens(o, "o", vv, _BF16, lead, dev), _ptr(o)
    with _on(dev):
        st = lib.gnorm_delta_step(ctypes.byref(d), _stream(stream, dev))
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
            else do.contiguous()
        dfinal = None if dfinal is None else dfinal.contiguous()
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
        """(y, final_state) over whole sequences; gate: BF16, v's shape."""
        o, final = gated_delta_rule(q, k, v, g, beta, scale=scale, cu_seqlens=cu_seqlens,
                                    initial_state=initial_state)
        return gated_rmsnorm(o, gate, self.weight, self.eps), final

    def step(self, q, k, v, g, beta, gate, state, *, slots=None, scale=None):
        """y for one token of each sequence; ``state`` is updated in place (no gradients)."""
        with torch.no_grad():
            o = gnorm_delta_step(q, k, v, g, beta, state, slots=slots, scale=scale)
            return gated_rmsnorm(o, gate, self.weight, self.eps)
