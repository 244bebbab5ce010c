"""Gradients written side by side into one wider buffer where the heads are grouped, so that a row
of dv is wider than one of dq (GPU): the same bits as in tensors of their own, and what lies
between them stays.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn
    from test_delta_gpu import GRADS, call, make


@pytest.mark.parametrize("Hk,Hv,K,V", [(2, 4, 128, 128), (1, 3, 64, 128), (2, 2, 128, 64)])
def test_one_gradient_of_a_projection(Hk, Hv, K, V):
    x = make([150, 3], Hk, Hv, K, V, state=True, tail=2)
    ref = call(x)
    n, w = 155, dict(dq=Hk * K, dk=Hk * K, dv=Hv * V)
    wide = torch.full((n, sum(w.values()) + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    narrow = torch.full((n, 2 * Hv + 1), 9.0, device="cuda")
    out, at = {}, 0
    for name, cols in w.items():
        out[name] = wide[:, at:at + cols].unflatten(1, (-1, V if name == "dv" else K))
        at += cols
    out["dg"], out["dbeta"] = narrow[:, :Hv], narrow[:, Hv:2 * Hv]
    got = call(x, **out)
    for name in GRADS:
        if name == "dS0":
            assert torch.equal(got[name], ref[name])
        else:
            assert got[name].data_ptr() == out[name].data_ptr()
            assert torch.equal(got[name][:153], ref[name][:153]), name
    assert bool((wide[:153, at:] == 9.0).all()) and bool((wide[153:] == 9.0).all())
    assert bool((narrow[:153, 2 * Hv:] == 9.0).all()) and bool((narrow[153:] == 9.0).all())
