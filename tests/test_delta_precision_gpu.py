"""What the gated delta rule holds in FP32 (states, dS0, dbeta, dg, and dv before it is rounded),
and sequences of six chunks in every kernel (GPU).

Norm-wise tolerance of the FP32 results, from the arithmetic.  Every operand that is not exact in
BF16 is in three BF16 parts, each off by half a step, 2^-8 of what the one before has left: 2^-24.
The six products of two such operands that are taken leave out terms of 2^-24.  What remains are
the sums: an accumulator takes 16 terms of the reduction at a time, 128 of them in three parts are
24 steps, and a step is off by at most 2^-23 of the sum (tensor cores cut, they do not round): 24
steps independent of each other are sqrt(24) 2^-23 = 5.8e-7 of a product's norm.  From a state to
the next there are three products in a row, in quadrature 1.0e-6; dg has one more behind them, and
1.2e-6.  With keys of unit length the steps enlarge no error of an earlier chunk, and the decay
takes it away as it takes the state: 1.5e-6 for all of them.  With two parts an operand is off by
up to 2^-16 = 1.5e-5; a state was 3e-6 of its norm off and dg 2e-6 to 3e-6, which this does not
let pass.

dbeta_t and dg_t are sums of many terms that can take each other back; their errors are compared
with the root of the sum of the terms' squares.  dv is rounded to BF16, at most 2^-8 relative, and
its FP32 value is off by the tolerance above.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from test_delta_gpu import call, check, close, make, recurrence

THREE_PARTS = 1.5e-6


def off(got, ref, size=None):
    """The error's norm relative to the reference's, or to that of `size`."""
    return float((got.double() - ref).norm() / (ref if size is None else size).norm())


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# Which kernels run (K, V, key heads, value heads, lengths): strips of 16 columns, one or two an SM;
# 32 columns of a head per CTA; a whole head per CTA, of one length and packed.
KERNELS = {
    "strip": (128, 128, 2, 4, [330]),
    "strip of 64": (64, 64, 2, 2, [330]),
    "two strips": (64, 128, 4, 24, [330]),
    "columns": (128, 128, 4, 24, [330]),
    "whole heads": (128, 128, 4, 40, [330]),
    "whole heads of K = 64": (64, 128, 4, 40, [330]),
    "whole heads packed": (128, 128, 2, 8, [330] + [1, 64, 65, 0, 3, 17] * 3 + [384]),
}


def which(K, V, Hv, B):
    """The forward's kernel for a call with these heads, by the rule that the library documents."""
    heads = Hv * B
    if V == 128 and (heads > sms() if B > 1 else 4 * heads > sms()):
        return "whole heads"
    if V // 16 * heads <= sms():
        return "strip"
    return "columns" if K == 128 else "two strips"


@pytest.mark.parametrize("name", KERNELS)
def test_fp32_results(name):
    K, V, Hk, Hv, lens = KERNELS[name]
    assert name.startswith(which(K, V, Hv, len(lens)))
    x = make(lens, Hk, Hv, K, V, state=True, decay=0.1, seed=len(name))
    got, ref = call(x), recurrence(x)
    assert off(got["S"], ref["S"]) <= THREE_PARTS
    assert off(got["dS0"], ref["dS0"]) <= THREE_PARTS
    for n in ("dbeta", "dg"):
        assert off(got[n], ref[n], ref["size"][n]) <= THREE_PARTS, n
    err = (got["dv"].double() - ref["dv"]).abs() - 2.0 ** -8 * ref["dv"].abs()
    assert float(err.clamp(min=0).norm() / ref["dv"].norm()) <= THREE_PARTS


@pytest.mark.parametrize("Hv", [24, 40])
@pytest.mark.parametrize("T", [321, 384])
def test_six_chunks(T, Hv):
    """The stages of the columns' and the whole heads' kernels in their second phase and after."""
    assert which(128, 128, Hv, 1) == ("columns" if Hv == 24 else "whole heads")
    check(make([T], 8, Hv, 128, 128, state=True, seed=T + Hv))


def test_many_chunks_of_some_heads():
    """Two phases more often than that; states against those of a call per chunk."""
    import gated_norm_b200 as gn

    for Hv in (24, 40):
        x = make([64 * 20], 4, Hv, 128, 128, state=True, decay=0.1)
        names = ("q", "k", "v", "g", "beta")
        o, S = gn.gnorm_delta_fwd(*(x[n] for n in names), scale=x["scale"], initial_state=x["S0"],
                                  output_final_state=True)
        S1, parts = x["S0"], []
        for t in range(0, 64 * 20, 64):
            p, S1 = gn.gnorm_delta_fwd(*(x[n][t:t + 64] for n in names), scale=x["scale"],
                                       initial_state=S1, output_final_state=True)
            parts.append(p)
        assert torch.equal(S, S1) and torch.equal(o, torch.cat(parts))
    assert gn.gnorm_device_error(reset=True) == 0


def test_the_backward_scan_in_two_waves():
    """More strips than SMs in the backward (one strip a CTA there): 24 heads of 128 columns."""
    x = make([200], 24, 24, 128, 128, decay=0.1)
    assert 24 * 8 > sms()
    got, ref = call(x), recurrence(x)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        close(got[n], ref[n], n, size=ref["size"])
