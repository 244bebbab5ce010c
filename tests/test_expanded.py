"""Expanded tensors (stride 0: one row, token or slot in the place of many) are refused on the
host, inputs and outputs alike, before anything is launched: a descriptor's stride of 0 means
packed, and rows behind the one that is there must not be read or written.  One row alone has no
stride and is accepted; a broadcast input made contiguous gets the gradient of its base.
"""
from __future__ import annotations

import pytest
import torch

import gated_norm_b200 as gn

SHARED = "share memory"


def one(*shape, dtype=torch.bfloat16, device="cpu"):
    """A tensor of this shape whose rows (the first dimension) are one and the same."""
    return torch.zeros((1,) + shape[1:], dtype=dtype, device=device).expand(shape)


def norm_calls(device):
    """Calls of the norms with one expanded argument each."""
    M, N = 6, 64
    x = torch.zeros(M, N, dtype=torch.bfloat16, device=device)
    w, st = torch.ones(N, device=device), torch.ones(M, device=device)
    e = one(M, N, device=device)
    e32 = one(M, N, dtype=torch.float32, device=device)
    yield "fwd x", lambda: gn.gnorm_fwd(e, x, w)
    yield "bwd x", lambda: gn.gnorm_bwd(x, e, x, w, st)
    yield "block a", lambda: gn.gnorm_block_fwd(e, x, w, w)
    yield "block_bwd a", lambda: gn.gnorm_block_bwd(None, x, e, x, w, w, st, st)
    if device == "cpu":  # whose other arguments come after the first one's device
        return
    yield "bwd dy", lambda: gn.gnorm_bwd(e, x, x, w, st)
    yield "block_bwd dz", lambda: gn.gnorm_block_bwd(None, e, x, x, w, w, st, st)
    yield "fwd g", lambda: gn.gnorm_fwd(x, e, w)
    yield "fwd y", lambda: gn.gnorm_fwd(x, x, w, y=e)
    yield "bwd dx", lambda: gn.gnorm_bwd(x, x, x, w, st, dx=e)
    yield "function g", lambda: gn.gated_rmsnorm(x, e, w)
    yield "block r", lambda: gn.gnorm_block_fwd(x, e, w, w)
    yield "block r fp32", lambda: gn.gnorm_block_fwd(x, e32, w, w)
    yield "block g", lambda: gn.gnorm_block_fwd(x, x, w, w, g=e)
    yield "block h", lambda: gn.gnorm_block_fwd(x, x, w, w, h=e)
    yield "block z", lambda: gn.gnorm_block_fwd(x, x, w, w, z=e)
    yield "block_bwd dh", lambda: gn.gnorm_block_bwd(e, x, x, x, w, w, st, st)
    yield "block_bwd r", lambda: gn.gnorm_block_bwd(x, x, x, e, w, w, st, st)
    for n in ("da", "dr", "dg"):
        yield "block_bwd " + n, lambda n=n: gn.gnorm_block_bwd(x, x, x, x, w, w, st, st, g=x, **{n: e})
    yield "block function", lambda: gn.block_rmsnorm(x, x, w, w, g=e)


def delta_calls(device):
    Hk, Hv, D = 1, 2, 64
    for lead in ((5,), (2, 5), (5, 1)):
        def full(heads, *tail, dtype=torch.bfloat16):
            return torch.zeros(*lead, heads, *tail, dtype=dtype, device=device)

        def same(t):  # every token the first one
            first = t[(slice(0, 1),) * len(lead)]
            return first.expand(t.shape)

        f = torch.float32
        a = dict(q=full(Hk, D), k=full(Hk, D), v=full(Hv, D), g=full(Hv, dtype=f),
                 beta=full(Hv, dtype=f))
        o = full(Hv, D)
        yield f"delta q {lead}", lambda a=a, s=same: gn.gnorm_delta_fwd(**{**a, "q": s(a["q"])})
        if device == "cpu":
            continue
        for n in ("k", "v", "g", "beta"):
            b = {**a, n: same(a[n])}
            yield f"delta {n} {lead}", lambda b=b: gn.gnorm_delta_fwd(**b)
            yield f"delta_bwd {n} {lead}", lambda b=b, o=o: gn.gnorm_delta_bwd(o, **b)
            yield f"rule {n} {lead}", lambda b=b: gn.gated_delta_rule(**b)
        yield f"delta o {lead}", lambda a=a, o=o, s=same: gn.gnorm_delta_fwd(**a, o=s(o))
        yield f"delta_bwd do {lead}", lambda a=a, o=o, s=same: gn.gnorm_delta_bwd(s(o), **a)
        for n in ("q", "k", "v", "g", "beta"):
            yield (f"delta_bwd d{n} {lead}", lambda a=a, o=o, s=same, n=n:
                   gn.gnorm_delta_bwd(o, **a, **{"d" + n: s(a[n])}))
        if len(lead) > 1:
            continue
        pool = torch.zeros(7, Hv, D, D, device=device)
        slots = torch.arange(5, dtype=torch.int32, device=device)
        for n in a:
            b = {**a, n: same(a[n])}
            yield "step " + n, lambda b=b: gn.gnorm_delta_step(**b, state=pool)
        yield "step o", lambda a=a, o=o, s=same: gn.gnorm_delta_step(**a, state=pool, o=s(o))
        yield "step state", lambda a=a: gn.gnorm_delta_step(**a, state=pool[:1].expand(7, Hv, D, D))
        yield "step state, slots", lambda a=a: gn.gnorm_delta_step(
            **a, state=pool[:1].expand(7, Hv, D, D), slots=slots)


def check_refused(calls):
    done = 0
    for name, call in calls:
        with pytest.raises(ValueError, match=SHARED):
            call()
            pytest.fail(name)
        done += 1
    return done


def test_refused_on_the_host():
    assert check_refused(norm_calls("cpu")) == 4
    assert check_refused(delta_calls("cpu")) == 3


@pytest.mark.gpu
def test_refused():
    assert check_refused(norm_calls("cuda")) > 15
    assert check_refused(delta_calls("cuda")) > 60
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_one_row_has_no_stride():
    """An expanded dimension of one row, token or slot is just that row."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rand(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    x, g, w = rand(1, 256).bfloat16(), rand(1, 256).bfloat16(), torch.ones(256, device="cuda")
    got = gn.gnorm_block_fwd(x.expand(1, 256), x, w, w, g=g.expand(1, 256))
    for p, q in zip(got, gn.gnorm_block_fwd(x, x, w, w, g=g)):
        assert torch.equal(p, q)
    a = [rand(1, 2, 64).bfloat16() for _ in range(3)] + [-rand(1, 2).abs(), rand(1, 2).sigmoid()]
    wide = [t.as_strided(t.shape, (0,) + t.stride()[1:]) for t in a]
    for p, q in zip(gn.gnorm_delta_fwd(*wide, output_final_state=True),
                    gn.gnorm_delta_fwd(*a, output_final_state=True)):
        assert torch.equal(p, q)
    pool = rand(1, 2, 64, 64)
    p1, p2 = pool.clone(), pool.clone()
    assert torch.equal(gn.gnorm_delta_step(*wide, p1.expand(1, 2, 64, 64)), gn.gnorm_delta_step(*a, p2))
    assert torch.equal(p1, p2)


@pytest.mark.gpu
def test_gradient_of_a_broadcast_input():
    """A decay and a step size per head, one for all tokens, through contiguous(): their gradients
    are the sums over the tokens of the full tensors'."""
    T, Hv = 130, 3
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rand(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    k = torch.nn.functional.normalize(rand(T, Hv, 64), dim=-1).bfloat16()
    q, v, do = (rand(T, Hv, 64).bfloat16() for _ in range(3))
    g = (-rand(Hv).abs()).requires_grad_()
    beta = rand(Hv).sigmoid().requires_grad_()
    o, _ = gn.gated_delta_rule(q, k, v, g.expand(T, Hv).contiguous(), beta.expand(T, Hv).contiguous())
    o.backward(do)
    full = gn.gnorm_delta_bwd(do, q, k, v, g.detach().repeat(T, 1), beta.detach().repeat(T, 1))
    assert torch.equal(g.grad, full[3].sum(0)) and torch.equal(beta.grad, full[4].sum(0))
