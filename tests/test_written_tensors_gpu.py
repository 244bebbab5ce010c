"""Tensors of the caller's that a call writes (the pool of states, outputs that are passed in) are
known to autograd as changed, so that a graph which has saved one raises in its backward instead
of taking the new values for the old (GPU).
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn
    from test_delta_gpu import make, step, step_case


def test_a_pool_stepped_before_the_backward():
    x = step_case(3, 1, 2, 64, 64, 3)
    pool = x["pool"].clone()
    v = torch.randn(3, 4, 2, 64, device="cuda").bfloat16().requires_grad_()
    z = torch.zeros(3, 4, 2, device="cuda")
    k = torch.nn.functional.normalize(torch.randn(3, 4, 1, 64, device="cuda"), dim=-1).bfloat16()
    for touched in (False, True):
        o, _ = gn.gated_delta_rule(k, k, v, z, z + 0.5, initial_state=pool)
        if touched:
            step(x, pool, slots=x["slots"])
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                o.sum().backward()
        else:
            o.sum().backward()


def bumps(call, *tensors):
    """Which of the tensors the call has left with another version."""
    before = [t._version for t in tensors]
    call()
    return [t._version != b for t, b in zip(tensors, before)]


def test_written_and_read():
    x = make([70], 1, 2, 64, 64, state=True)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    assert bumps(lambda: gn.gnorm_delta_fwd(*a, initial_state=x["S0"], o=o, final_state=S),
                 o, S, x["S0"], *a) == [True] * 2 + [False] * 6
    out = {"d" + n: torch.empty_like(x[n]) for n in ("q", "k", "v", "g", "beta")}
    dS0 = torch.empty_like(S)
    assert bumps(lambda: gn.gnorm_delta_bwd(x["do"], *a, initial_state=x["S0"], dinitial_state=dS0, **out),
                 *out.values(), dS0, x["do"], x["S0"], *a) == [True] * 6 + [False] * 7
    y = step_case(3, 1, 2, 64, 64, 3)
    o1 = torch.empty_like(y["v"])
    assert bumps(lambda: step(y, y["pool"], slots=y["slots"], o=o1),
                 y["pool"], o1, y["q"], y["slots"]) == [True, True, False, False]
    r = torch.randn(5, 64, device="cuda").bfloat16()
    w, al = torch.ones(64, device="cuda"), torch.ones(1, device="cuda")
    fwd = [torch.empty_like(r), torch.empty_like(r), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")]
    names = ("h", "z", "rstd1", "rstd2")
    assert bumps(lambda: gn.gnorm_block_fwd(r, r, w, w, g=r, alpha=al, **dict(zip(names, fwd))),
                 *fwd, r, w, al) == [True] * 4 + [False] * 3
    bwd = [torch.empty_like(r) for _ in range(3)] + [torch.empty_like(w), torch.empty_like(w), torch.empty_like(al)]
    names = ("da", "dr", "dg", "dw1", "dw2", "dalpha")
    assert bumps(lambda: gn.gnorm_block_bwd(r, r, r, r, w, w, fwd[2], fwd[3], g=r, alpha=al, dw_fp32=True,
                                            **dict(zip(names, bwd))),
                 *bwd, r, w, al, *fwd) == [True] * 6 + [False] * 7


def test_refused_calls_and_inference_tensors():
    x = step_case(3, 1, 2, 64, 64, 5)
    pool = x["pool"].clone()
    version = pool._version
    with pytest.raises(gn.GnormError):  # more rows than slots
        step(x, pool[:2])
    assert pool._version == version
    with torch.inference_mode():
        state = x["pool"].clone()
        o = step(x, state, slots=x["slots"])
    o2 = step(x, pool, slots=x["slots"])
    assert torch.equal(o, o2) and torch.equal(state, pool)
    step(x, state, slots=x["slots"])  # of a pool made in inference mode, outside of it
    step(x, pool, slots=x["slots"])
    assert torch.equal(state, pool)
