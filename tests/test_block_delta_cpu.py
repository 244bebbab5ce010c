"""The block norm and the gated delta rule without a GPU: the C entry points refuse bad
arguments before any CUDA call, workspace sizes, and the binding's checks of host tensors.
No kernel is launched.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_norm_b200 as gn
from gated_norm_b200._lib import (GNORM_ERR_ALIAS, GNORM_ERR_ALIGN, GNORM_ERR_ARG, GNORM_ERR_NULL,
                                  GNORM_ERR_SHAPE, GNORM_ERR_WORKSPACE, GNORM_OK,
                                  GnormBlockBwdDesc, GnormBlockFwdDesc, GnormDeltaBwdDesc,
                                  GnormDeltaFwdDesc, GnormDeltaIn, GnormDeltaStepDesc, lib)

MB = 1 << 20


class Places:
    """Made-up device addresses, far enough apart not to overlap; nothing reads them."""

    def __init__(self):
        self.at = 1 << 40

    def __call__(self):
        self.at += 1 << 34
        return self.at


def call(fn, desc):
    return fn(ctypes.byref(desc), None)


# --------------------------------------------------------------------------- block norm

def block_fwd(**kw):
    p = Places()
    d = GnormBlockFwdDesc(a=p(), r=p(), g=p(), w1=p(), w2=p(), alpha=p(), eps1=1e-6, eps2=1e-6,
                          h=p(), z=p(), rstd1=p(), rstd2=p(), M=16, N=256)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(N=250), GNORM_ERR_SHAPE), (dict(N=0), GNORM_ERR_SHAPE), (dict(N=16392), GNORM_ERR_SHAPE),
    (dict(M=-1), GNORM_ERR_SHAPE), (dict(eps1=-1.0), GNORM_ERR_ARG),
    (dict(eps2=float("nan")), GNORM_ERR_ARG), (dict(lda=128), GNORM_ERR_SHAPE),
    (dict(ldz=260), GNORM_ERR_ALIGN), (dict(a=None), GNORM_ERR_NULL), (dict(w2=None), GNORM_ERR_NULL),
    (dict(rstd2=None), GNORM_ERR_NULL), (dict(alpha=4097), GNORM_ERR_ALIGN),
    (dict(r=(1 << 50) + 8), GNORM_ERR_ALIGN), (dict(M=0, a=None, h=None), GNORM_OK)])
def test_block_fwd_refuses(kw, status):
    assert call(lib.gnorm_block_fwd, block_fwd(**kw)) == status


def test_block_aliases():
    d = block_fwd()
    d.h = d.r
    assert call(lib.gnorm_block_fwd, d) == GNORM_ERR_ALIAS
    d = block_fwd()
    d.z = d.a + 16 * 256 * 2 - 16  # the last 16 bytes of a
    assert call(lib.gnorm_block_fwd, d) == GNORM_ERR_ALIAS
    d = block_fwd()
    d.rstd2 = d.rstd1 + 4
    assert call(lib.gnorm_block_fwd, d) == GNORM_ERR_ALIAS
    assert lib.gnorm_block_fwd(None, None) == GNORM_ERR_NULL


def block_bwd(**kw):
    p = Places()
    d = GnormBlockBwdDesc(dh=p(), dz=p(), a=p(), r=p(), g=p(), w1=p(), w2=p(), alpha=p(), rstd1=p(),
                          rstd2=p(), da=p(), dr=p(), dg=p(), dw1=p(), dw2=p(), dalpha=p(), M=16,
                          N=256, workspace=p(), workspace_bytes=MB)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(N=12), GNORM_ERR_SHAPE), (dict(dz=None), GNORM_ERR_NULL), (dict(dg=None), GNORM_ERR_NULL),
    (dict(g=None), GNORM_ERR_NULL), (dict(alpha=None), GNORM_ERR_NULL), (dict(dw1=None), GNORM_ERR_NULL),
    (dict(lddr=100), GNORM_ERR_SHAPE), (dict(dw2=(1 << 50) + 4), GNORM_ERR_ALIGN)])
def test_block_bwd_refuses(kw, status):
    assert call(lib.gnorm_block_bwd, block_bwd(**kw)) == status


def test_block_bwd_aliases():
    d = block_bwd()
    d.da = d.dz
    assert call(lib.gnorm_block_bwd, d) == GNORM_ERR_ALIAS
    d = block_bwd()
    d.workspace = d.dw1
    assert call(lib.gnorm_block_bwd, d) == GNORM_ERR_ALIAS


# --------------------------------------------------------------------------- delta rule

def delta_in(p, **kw):
    d = GnormDeltaIn(q=p(), k=p(), v=p(), g=p(), beta=p(), beta_fp32=1, cu_seqlens=p(), B=3, T=200,
                     Hk=2, Hv=4, K=128, V=64, scale=0.1, initial_state=p())
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def delta_fwd(top=None, **kw):
    p = Places()
    d = GnormDeltaFwdDesc(o=p(), final_state=p(), workspace=p(), workspace_bytes=64 * MB)
    setattr(d, "in", delta_in(p, **kw))
    for k, v in (top or {}).items():
        setattr(d, k, v)
    return d


IN_REFUSALS = [
    (dict(K=32), GNORM_ERR_SHAPE), (dict(V=256), GNORM_ERR_SHAPE), (dict(Hv=3), GNORM_ERR_SHAPE),
    (dict(Hk=0), GNORM_ERR_SHAPE), (dict(Hv=65536), GNORM_ERR_SHAPE), (dict(T=-1), GNORM_ERR_SHAPE),
    (dict(T=1 << 31), GNORM_ERR_SHAPE), (dict(B=65536), GNORM_ERR_SHAPE),
    (dict(B=0), GNORM_ERR_SHAPE), (dict(cu_seqlens=None), GNORM_ERR_SHAPE),  # 200 tokens, 3 sequences
    (dict(scale=float("inf")), GNORM_ERR_ARG), (dict(ldq=128), GNORM_ERR_SHAPE),
    (dict(ldv=260), GNORM_ERR_ALIGN), (dict(ldg=3), GNORM_ERR_SHAPE), (dict(q=None), GNORM_ERR_NULL),
    (dict(beta=None), GNORM_ERR_NULL), (dict(k=(1 << 50) + 8), GNORM_ERR_ALIGN),
    (dict(beta=(1 << 50) + 2), GNORM_ERR_ALIGN), (dict(initial_state=(1 << 50) + 4), GNORM_ERR_ALIGN)]


@pytest.mark.parametrize("kw,status", IN_REFUSALS)
def test_delta_refuses(kw, status):
    assert call(lib.gnorm_delta_fwd, delta_fwd(**kw)) == status
    assert call(lib.gnorm_delta_bwd, delta_bwd(**kw)) == status


@pytest.mark.parametrize("top,status", [
    (dict(o=None), GNORM_ERR_NULL), (dict(ldo=8), GNORM_ERR_SHAPE), (dict(o=(1 << 50) + 8), GNORM_ERR_ALIGN),
    (dict(workspace=None), GNORM_ERR_WORKSPACE), (dict(workspace_bytes=4096), GNORM_ERR_WORKSPACE),
    (dict(workspace=(1 << 50) + 64), GNORM_ERR_WORKSPACE)])
def test_delta_fwd_refuses(top, status):
    assert call(lib.gnorm_delta_fwd, delta_fwd(top)) == status


def test_delta_aliases():
    d = delta_fwd()
    d.o = getattr(d, "in").v
    assert call(lib.gnorm_delta_fwd, d) == GNORM_ERR_ALIAS
    d = delta_fwd()
    d.final_state = getattr(d, "in").initial_state
    assert call(lib.gnorm_delta_fwd, d) == GNORM_ERR_ALIAS
    d = delta_fwd()
    d.workspace = d.final_state
    assert call(lib.gnorm_delta_fwd, d) == GNORM_ERR_ALIAS
    d = delta_bwd()
    d.dk = d.dq
    assert call(lib.gnorm_delta_bwd, d) == GNORM_ERR_ALIAS
    # nothing to do: no sequences, no tokens
    assert call(lib.gnorm_delta_fwd, delta_fwd(dict(o=None), B=0, T=0, cu_seqlens=None)) == GNORM_OK


def delta_bwd(top=None, **kw):
    p = Places()
    d = GnormDeltaBwdDesc(d_o=p(), dfinal_state=p(), dq=p(), dk=p(), dv=p(), dg=p(), dbeta=p(),
                          dinitial_state=p(), workspace=p(), workspace_bytes=64 * MB)
    setattr(d, "in", delta_in(p, **kw))
    for k, v in (top or {}).items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("top,status", [
    (dict(d_o=None), GNORM_ERR_NULL), (dict(dbeta=None), GNORM_ERR_NULL),
    (dict(lddk=4), GNORM_ERR_SHAPE), (dict(lddv=257), GNORM_ERR_ALIGN),
    (dict(dg=(1 << 50) + 2), GNORM_ERR_ALIGN), (dict(workspace_bytes=1 << 18), GNORM_ERR_WORKSPACE)])
def test_delta_bwd_refuses(top, status):
    assert call(lib.gnorm_delta_bwd, delta_bwd(top)) == status


def test_delta_workspace_bytes():
    for K, V in ((64, 64), (64, 128), (128, 64), (128, 128)):
        last = 0
        for T in (0, 1, 64, 1000, 100000):
            fwd = gn.gnorm_delta_workspace_bytes(T, 3, 4, K, V)
            bwd = gn.gnorm_delta_workspace_bytes(T, 3, 4, K, V, True)
            slots = T // 64 + 4
            assert fwd % 256 == 0 and fwd >= slots * 4 * 6 * 5120
            assert bwd >= fwd + slots * 4 * (8 * K * V + 3 * 64 * V * 2 + 64 * V * 2)
            assert fwd >= last
            last = fwd
    for bad in ((-1, 1, 4, 128, 128), (64, 70000, 4, 128, 128), (64, 1, 0, 128, 128),
                (64, 1, 4, 96, 128), (64, 1, 4, 128, 256), (1 << 31, 1, 4, 128, 128)):
        assert gn.gnorm_delta_workspace_bytes(*bad) == 0


def step(**kw):
    p = Places()
    d = GnormDeltaStepDesc(q=p(), k=p(), v=p(), g=p(), beta=p(), B=5, Hk=2, Hv=4, K=128, V=128,
                           scale=0.1, state=p(), pool=8, slots=p(), o=p())
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(K=16), GNORM_ERR_SHAPE), (dict(Hv=5), GNORM_ERR_SHAPE), (dict(B=-1), GNORM_ERR_SHAPE),
    (dict(pool=-1), GNORM_ERR_SHAPE), (dict(slots=None, pool=4), GNORM_ERR_SHAPE),
    (dict(scale=float("nan")), GNORM_ERR_ARG), (dict(ldstate=1000), GNORM_ERR_SHAPE),
    (dict(ldstate=4 * 128 * 128 + 2), GNORM_ERR_ALIGN), (dict(ldv=514), GNORM_ERR_ALIGN),
    (dict(q=None), GNORM_ERR_NULL), (dict(state=None), GNORM_ERR_NULL),
    (dict(state=(1 << 50) + 8), GNORM_ERR_ALIGN), (dict(o=(1 << 50) + 4), GNORM_ERR_ALIGN),
    (dict(B=0, q=None), GNORM_OK)])
def test_step_refuses(kw, status):
    assert call(lib.gnorm_delta_step, step(**kw)) == status


def test_step_aliases():
    d = step()
    d.o = d.v
    assert call(lib.gnorm_delta_step, d) == GNORM_ERR_ALIAS
    d = step()
    d.o = d.state + 64
    assert call(lib.gnorm_delta_step, d) == GNORM_ERR_ALIAS


# ---------------------------------------------------------------------------- the binding

def test_binding_rejects_host_tensors():
    def bf16(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    a, w = bf16(4, 128), torch.ones(128)
    with pytest.raises(ValueError, match="CUDA"):
        gn.gnorm_block_fwd(a, a, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        gn.gnorm_block_bwd(a, a, a, a, w, w, torch.ones(4), torch.ones(4))
    q, g = bf16(4, 2, 64), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        gn.gnorm_delta_fwd(q, q, q, g, g)
    with pytest.raises(ValueError, match="CUDA"):
        gn.gnorm_delta_bwd(q, q, q, q, g, g)
    with pytest.raises(ValueError, match="CUDA"):
        gn.gnorm_delta_step(q, q, q, g, g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError):
        gn.gnorm_delta_fwd(q[0], q[0], q[0], g, g)  # no token dimension
    with pytest.raises(TypeError):
        gn.gnorm_delta_fwd(q.float(), q, q, g, g)
