"""The gated delta rule (gnorm_delta_fwd / gnorm_delta_bwd / gnorm_delta_step) against the
recurrence token by token in FP64, and its adjoint (GPU).

Tolerances, from the arithmetic: a value split in two BF16 values keeps it to 2^-16 relative
(two half steps of 2^-8), and a product of two split values leaves out lo x lo, another 2^-16;
the way from the inputs to a state, an output or a gradient goes through at most four such
products a chunk, and with keys of unit length the steps from chunk to chunk do not enlarge an
error.  Every output is so within 2^-14 = 4 x 2^-16 of the exact value relative to the RMS of
its head's vector or its own size; an output in BF16 adds half a step, 2^-8 relative.  The
gradients of k, q, g and beta are sums over V columns, all value heads of a key head or a whole
state, dk_t = sum (dS u - S du beta), dq_t = sum S do, dg_t = <e^g S, d(e^g S)>, dbeta_t =
<w, du>, and o_t = scale sum_j e^(..) (q_t k_j) u_j one over the tokens before; they can be much
smaller than their terms (the first and last tokens of a sequence, a sum of 16384 terms of
either sign, a key that comes again and again and whose u_j take each other back).  Each term carries the relative error of its factors, the
errors are roundings independent of each other, so the sum's error is 2^-14 of the root of the
sum of the terms' squares, and that takes the place of the RMS where it is larger.  The single step works in FP32: sums of 128 terms, 1e-5.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn

SPLIT = 2.0 ** -14
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def make(lens, Hk, Hv, K, V, *, state=False, beta=torch.float32, seed=0, tail=0, decay=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    T, B = sum(lens) + tail, len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    norm = torch.nn.functional.normalize
    return dict(q=norm(rand(T, Hk, K), dim=-1).bfloat16(),
                k=norm(rand(T, Hk, K) + 0.5 * rand(1, Hk, K), dim=-1).bfloat16(),
                v=rand(T, Hv, V).bfloat16(),
                g=-decay * torch.nn.functional.softplus(rand(T, Hv) - 2.0),
                beta=torch.sigmoid(rand(T, Hv)).to(beta),
                S0=0.3 * rand(B, Hv, K, V) if state else None,
                cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), lens=list(lens),
                scale=K ** -0.5, do=rand(T, Hv, V).bfloat16(),
                dS=0.1 * rand(B, Hv, K, V) if state else None)


def recurrence(x, grads=True):
    """o, the final states and the gradients, from the definition in FP64."""
    r = x["v"].shape[1] // x["q"].shape[1]
    names = ("q", "k", "v", "g", "beta", "S0")
    leaf = {n: None if x[n] is None else x[n].double().requires_grad_(grads) for n in names}
    q, k = (leaf[n].repeat_interleave(r, 1) for n in ("q", "k"))
    v, w, beta = leaf["v"], torch.exp(leaf["g"]), leaf["beta"]
    T, Hv, V = v.shape
    K = q.shape[2]
    outs, states = [], []
    inner = []  # per token: the decayed state, w, u and the new state
    t = 0
    for b, n in enumerate(x["lens"]):
        S = leaf["S0"][b] if leaf["S0"] is not None else \
            torch.zeros(Hv, K, V, dtype=torch.float64, device="cuda")
        for _ in range(n):
            Sd = w[t][:, None, None] * S
            e = v[t] - (k[t][:, :, None] * Sd).sum(1)
            u = beta[t][:, None] * e
            S = Sd + k[t][:, :, None] * u[:, None, :]
            inner.append((Sd, e, u, S))
            outs.append(x["scale"] * (q[t][:, :, None] * S).sum(1))
            t += 1
        states.append(S)
    o = torch.stack(outs) if outs else torch.zeros(0, Hv, V, dtype=torch.float64, device="cuda")
    S = torch.stack(states)
    out = dict(o=o.detach(), S=S.detach(), size={})
    # the roots of the sums of the squares of the terms of o, over all tokens before
    with torch.no_grad():
        rows, t = [], 0
        for b, n in enumerate(x["lens"]):
            s2 = leaf["S0"][b].square() if leaf["S0"] is not None else \
                torch.zeros(Hv, K, V, dtype=torch.float64, device="cuda")
            before = torch.zeros(0, Hv, dtype=torch.float64, device="cuda")
            for i in range(n):
                s2, before = s2 * w[t + i][:, None, None] ** 2, before * w[t + i]
                before = torch.cat([before, torch.ones_like(w[:1])])
                coef = before * torch.einsum("hk,jhk->jh", q[t + i], k[t:t + i + 1])
                us = torch.stack([inner[t + j][2] for j in range(i + 1)]).detach()
                first = torch.einsum("hk,hkv->hv", q[t + i].square(), s2)
                rows.append(x["scale"] *
                            (first + (coef[..., None] * us).square().sum(0)).sqrt())
            t += n
        if rows:
            out["size"]["o"] = torch.stack(rows)
    if grads and t:
        ys, ds = [o], [x["do"][:t].double()]
        if x["dS"] is not None:
            ys, ds = ys + [S], ds + [x["dS"].double()]
        have = [n for n in names if leaf[n] is not None]
        deep = [m for Sd, _, u, S in inner for m in (Sd, u, S) if m.requires_grad]
        ds = torch.autograd.grad(ys, [leaf[n] for n in have] + deep, ds, allow_unused=True)
        for n, d in zip(have, ds):
            out["d" + n] = d
        # the roots of the sums of the squares of the terms of dq, dk, dg and dbeta
        at = {id(m): d for m, d in zip(deep, ds[len(have):])}
        rows = {n: [] for n in ("dq", "dk", "dg", "dbeta")}
        for i, (Sd, e, u, S) in enumerate(inner):
            dSd, du, dS = (at.get(id(m)) if at.get(id(m)) is not None else torch.zeros_like(m)
                           for m in (Sd, u, S))
            rows["dg"].append((Sd * dSd).square().sum((1, 2)))
            rows["dbeta"].append((e * du).square().sum(1))
            rows["dq"].append((x["scale"] * S * x["do"][i].double()[:, None, :]).square().sum(2))
            rows["dk"].append(((dS * u[:, None, :]).square() +
                               (Sd * (beta[i][:, None] * du)[:, None, :]).square()).sum(2))
        for n, v in rows.items():
            v = torch.stack(v).detach()
            if n in ("dq", "dk"):  # over the value heads of a key head
                v = v.unflatten(1, (-1, r)).sum(2)
            out["size"][n] = v.sqrt()
    return out


def close(got, ref, name, tol=SPLIT, size=None):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    rms = ref.square().mean((-1, -2) if ref.dim() == 4 else -1, keepdim=True).sqrt()
    if size and name in size:
        rms = size[name] if name in ("dg", "dbeta") else torch.maximum(rms, size[name])
    err = (got.double() - ref).abs()
    half = torch.finfo(got.dtype).eps / 2 if got.dtype == torch.bfloat16 else 0.0
    lim = half * ref.abs() + tol * torch.maximum(rms, ref.abs()) + 1e-30
    assert bool((err <= lim).all()), (name, float((err / lim).max()))


def call(x, **kw):
    o, S = gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                              cu_seqlens=x["cu"], initial_state=x["S0"],
                              output_final_state=True)
    grads = gn.gnorm_delta_bwd(x["do"], x["q"], x["k"], x["v"], x["g"], x["beta"],
                               scale=x["scale"], cu_seqlens=x["cu"], initial_state=x["S0"],
                               dfinal_state=x["dS"], **kw)
    return dict(zip(("o", "S") + GRADS, (o, S) + grads))


def check(x, by_head=False):
    got, ref = call(x), recurrence(x)
    if by_head:
        ref["size"]["dv"] = ref["dv"].square().mean((0, 2), keepdim=True).sqrt()
        for n in ("dbeta", "dg"):
            ref["size"][n] = ref["size"][n].amax(0, keepdim=True)
    n = sum(x["lens"])
    for name, t in got.items():
        if t is None:
            assert name == "dS0" and x["S0"] is None
            continue
        if name not in ("S", "dS0"):
            assert not t[n:].any(), name  # behind the last sequence: zero
            t = t[:n]
        want = ref[name][:n] if name not in ("S", "dS0") else ref[name]
        close(t, want, name, size=ref["size"])
    return got


HEADS = [(128, 128, 2, 4), (64, 64, 3, 3), (64, 128, 1, 2), (128, 64, 2, 2)]


@pytest.mark.parametrize("K,V,Hk,Hv", HEADS)
@pytest.mark.parametrize("T", [1, 2, 15, 63, 64, 65, 129, 200])
def test_one_sequence(T, K, V, Hk, Hv):
    check(make([T], Hk, Hv, K, V, state=T % 2 == 1, seed=T,
               beta=torch.bfloat16 if T % 3 else torch.float32))


@pytest.mark.parametrize("K,V,Hk,Hv", HEADS)
@pytest.mark.parametrize("lens,tail", [([1, 64, 3, 65, 0, 130], 0), ([0, 0, 70], 5),
                                       ([63, 1, 1, 64, 128], 70), ([100, 0], 1)])
def test_packed_sequences(lens, tail, K, V, Hk, Hv):
    check(make(lens, Hk, Hv, K, V, state=True, tail=tail, seed=len(lens)))


def test_many_short_sequences():
    check(make([1 + i % 5 for i in range(150)], 1, 1, 64, 64, state=True))


def many_heads(seqs, Hv):
    """Enough sequences and heads for a whole head per SM (heads of 128 columns)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert seqs * Hv > sms
    return seqs, Hv


@pytest.mark.parametrize("K", [64, 128])
def test_whole_heads_packed(K):
    seqs, Hv = many_heads(40, 4)
    lens = [(1, 64, 0, 65, 130, 3, 63, 17)[i % 8] for i in range(seqs)]
    x = make(lens, 2, Hv, K, 128, state=True, tail=9, beta=torch.bfloat16)
    check(x)
    first = call(x)
    x["v"][200, 1] = float("nan")  # in one sequence, one head
    got = call(x)
    b = next(i for i in range(seqs) if sum(lens[:i + 1]) > 200)
    lo, hi = sum(lens[:b]), sum(lens[:b + 1])
    assert torch.equal(got["o"][:lo], first["o"][:lo]) and torch.equal(got["o"][hi:], first["o"][hi:])
    assert torch.equal(got["o"][:, [0, 2, 3]], first["o"][:, [0, 2, 3]])
    keep = [i for i in range(seqs) if i != b]
    assert torch.equal(got["S"][keep], first["S"][keep])


@pytest.mark.parametrize("K,L", [(128, 1), (64, 64), (128, 129)])
def test_whole_heads_of_one_length(K, L):
    """The batch form, without an initial state, on two streams at once and replayed."""
    B, Hv = many_heads(40, 4)
    x = make([L] * B, 1, Hv, K, 128)
    y = [x[n].unflatten(0, (B, L)) for n in ("q", "k", "v", "g", "beta")]
    o, S = gn.gnorm_delta_fwd(*y, output_final_state=True)
    ref = recurrence(x, grads=False)
    close(o.flatten(0, 1), ref["o"], "o", size=ref["size"])
    close(S, ref["S"], "S")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, S2 = gn.gnorm_delta_fwd(*y, output_final_state=True)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o4, S4 = gn.gnorm_delta_fwd(*y, output_final_state=True)
    o3, S3 = gn.gnorm_delta_fwd(*y, output_final_state=True)
    torch.cuda.current_stream().wait_stream(s)
    g.replay()
    torch.cuda.synchronize()
    for p, q in ((o2, S2), (o3, S3), (o4, S4)):
        assert torch.equal(p, o) and torch.equal(q, S)
    assert gn.gnorm_device_error(reset=True) == 0


def test_whole_heads_reset_and_repeat():
    seqs, Hv = many_heads(40, 4)
    x = make([70] * seqs, 1, Hv, 128, 128, state=True, decay=0.01)
    x["k"] = x["k"][:1].expand(70 * seqs, 1, 128).contiguous()
    x["beta"][:] = 0.9
    x["g"][30] = float("-inf")
    o, S = gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                              cu_seqlens=x["cu"], initial_state=x["S0"], output_final_state=True)
    ref = recurrence(dict(x, g=x["g"].clamp(min=-700.0)), grads=False)
    close(o, ref["o"], "o", size=ref["size"])
    close(S, ref["S"], "S")


def quarters(seqs, Hv, V, packed):
    """Heads of K = 128 that have 32 columns per CTA: more strips of 16 than SMs, and too few whole
    heads."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert V // 16 * Hv * seqs > sms and Hv * seqs * (1 if packed or V == 64 else 4) <= sms
    return Hv


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 129, 200])
def test_quarters_of_one_sequence(T):
    Hv = quarters(1, 24, 128, False)
    check(make([T], 8, Hv, 128, 128, state=T % 2 == 1, seed=T,
               beta=torch.bfloat16 if T % 3 else torch.float32))


@pytest.mark.parametrize("V", [64, 128])
def test_quarters_packed(V):
    lens = [65, 0, 130, 64, 1]
    Hv = quarters(len(lens), 8, V, True)
    x = make(lens, 2, Hv, 128, V, state=True, tail=70, seed=V)
    check(x)
    first = call(x)
    for n in ("q", "k", "v", "g", "beta"):
        x[n][260:] = float("nan")  # behind the last sequence
    x["v"][100, 1] = float("nan")  # in one sequence, one head
    x["S0"][3, 2, 5, 7] = float("inf")
    got = call(x)
    keep = list(range(65)) + [259]
    assert torch.equal(got["o"][keep], first["o"][keep])
    assert torch.equal(got["S"][[0, 1, 4]], first["S"][[0, 1, 4]])
    others = [0] + list(range(3, Hv))
    assert torch.equal(got["o"][:260, others], first["o"][:260, others])
    assert torch.equal(got["S"][:, others], first["S"][:, others])
    assert not bool(torch.isfinite(got["S"][2, 1]).all())


def test_quarters_reset_and_repeat():
    Hv = quarters(1, 20, 128, False)
    x = make([200], 1, Hv, 128, 128, state=True, decay=0.01)
    x["k"] = x["k"][:1].expand(200, 1, 128).contiguous()
    x["beta"][:] = 0.9
    x["g"][30] = float("-inf")
    x["g"][130] = torch.finfo(torch.float32).min
    o, S = gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                              cu_seqlens=x["cu"], initial_state=x["S0"], output_final_state=True)
    ref = recurrence(dict(x, g=x["g"].clamp(min=-700.0)), grads=False)
    close(o, ref["o"], "o", size=ref["size"])
    close(S, ref["S"], "S")


def test_quarters_streams_slices_and_replay():
    """Strided inputs and output, two streams at once, captured and replayed; what lies between
    the output's rows and behind the sequence stays."""
    T, Hv = 150, quarters(1, 24, 128, False)
    x = make([T], 8, Hv, 128, 128, state=True)
    args = lambda v: (x["q"], x["k"], v, x["g"], x["beta"])
    kw = dict(scale=x["scale"], initial_state=x["S0"], output_final_state=True)
    o, S = gn.gnorm_delta_fwd(*args(x["v"]), **kw)
    wide = torch.full((T, Hv * 128 + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + Hv * 128] = x["v"].reshape(T, -1)
    v = wide[:, 8:8 + Hv * 128].unflatten(1, (Hv, 128))
    cu = torch.tensor([0, 140], dtype=torch.int32, device="cuda")
    place = torch.full_like(wide, 7.0)
    o2, S2 = gn.gnorm_delta_fwd(*args(v), **kw, o=place[:, 8:8 + Hv * 128].unflatten(1, (Hv, 128)))
    assert torch.equal(o2, o) and torch.equal(S2, S)
    assert bool((place[:, :8] == 7.0).all()) and bool((place[:, 8 + Hv * 128:] == 7.0).all())
    part = torch.full_like(x["v"], 7.0)
    gn.gnorm_delta_fwd(*args(x["v"]), **kw, cu_seqlens=cu, o=part)
    assert torch.equal(part[:140], o[:140]) and bool((part[140:] == 7.0).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3, S3 = gn.gnorm_delta_fwd(*args(v), **kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o4, S4 = gn.gnorm_delta_fwd(*args(v), **kw)
    o5, S5 = gn.gnorm_delta_fwd(*args(x["v"]), **kw)
    torch.cuda.current_stream().wait_stream(s)
    g.replay()
    torch.cuda.synchronize()
    for a, b in ((o3, S3), (o4, S4), (o5, S5)):
        assert torch.equal(a, o) and torch.equal(b, S)
    assert gn.gnorm_device_error(reset=True) == 0


def test_many_heads_of_one_key_head():
    check(make([97], 1, 8, 128, 128))


@pytest.mark.parametrize("decay", [0.0, 0.01, 30.0])
def test_slow_and_fast_decay(decay):
    """No decay at all, and heads that forget within a token: no gradient loses its digits to
    terms that cancel."""
    check(make([257], 2, 2, 128, 128, state=True, decay=decay))


@pytest.mark.parametrize("reset", [float("-inf"), torch.finfo(torch.float32).min, -1000.0])
def test_full_reset(reset):
    """g of -inf (or so low that e^g is zero) starts the state anew: what follows equals a
    sequence of its own."""
    x = make([150], 2, 4, 128, 128, state=True)
    x["g"][70] = reset
    x["g"][99:101] = reset
    got, ref = call(x), recurrence(dict(x, g=x["g"].clamp(min=-700.0)))
    for name, t in got.items():
        assert bool(torch.isfinite(t).all()), name
        close(t, ref[name], name, size=ref["size"])
    assert not got["dg"][70].any() and not got["dg"][99:101].any()
    y = make([50], 2, 4, 128, 128)
    for n in ("q", "k", "v", "g", "beta"):
        y[n] = x[n][100:].contiguous()
    o, S = gn.gnorm_delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], scale=x["scale"],
                              output_final_state=True)
    ref = recurrence(dict(y, g=y["g"].clamp(min=-700.0)), grads=False)
    close(o, ref["o"], "o")
    close(S, ref["S"], "S")
    close(got["S"], ref["S"], "S")


def test_beta_zero_and_one():
    x = make([130], 2, 2, 64, 64, state=True)
    x["beta"][:40] = 0.0
    x["beta"][40:100] = 1.0
    check(x)


def test_repeated_keys():
    """The same key at every token: the triangular system at its least well conditioned.  dv is
    its solution, dv_t = beta_t sum_i T_ti dY_i over the chunk's tokens: where every key is the
    same, dY_i and dY_(i+1) differ by one row of do and T takes the differences, so a row's
    terms are as large as the head's rows, however small the row itself: they are compared with
    the head's RMS, and dbeta and dg, products with these rows, with the head's largest."""
    x = make([192], 1, 1, 128, 128, decay=0.01)
    x["k"] = x["k"][:1].expand(192, 1, 128).contiguous()
    x["beta"][:] = 0.9
    check(x, by_head=True)


def test_what_lies_behind_the_last_sequence():
    """Not read (NaN there changes nothing), zero in new outputs, left alone in given ones."""
    x = make([70, 30], 1, 2, 128, 64, state=True, tail=90)
    clean = call(x)
    for n in ("q", "k", "v", "g", "beta", "do"):
        x[n][100:] = float("nan")
    for n, t in call(x).items():
        assert torch.equal(t, clean[n]), n
    o = torch.full_like(x["v"], 7.0)
    gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                       cu_seqlens=x["cu"], initial_state=x["S0"], o=o)
    assert torch.equal(o[:100], clean["o"][:100]) and bool((o[100:] == 7.0).all())
    out = {n: torch.full_like(clean[n], 7.0) for n in GRADS[:5]}
    call(x, **out)
    for n, t in out.items():
        assert torch.equal(t[:100], clean[n][:100]) and bool((t[100:] == 7.0).all()), n


def test_non_finite_inputs_stay_in_their_sequence():
    x = make([70, 80, 66], 1, 2, 128, 128, state=True)
    clean = call(x)
    x["v"][140, 1] = float("nan")  # in the sequence's second chunk: the first stays clean
    x["S0"][1, 0, 3, 5] = float("inf")
    got = call(x)
    keep = list(range(70)) + list(range(150, 216))
    for n, t in got.items():
        if n in ("S", "dS0"):
            assert torch.equal(t[[0, 2]], clean[n][[0, 2]]), n
        else:
            assert torch.equal(t[keep], clean[n][keep]), n
    assert bool(torch.isnan(got["o"][141, 1]).any()) and bool(torch.isfinite(got["o"][133, 1]).all())


def test_batch_form():
    x = make([67, 67, 67], 2, 2, 64, 128, state=True)
    flat = call(x)
    y = {n: x[n].view(3, 67, *x[n].shape[1:]) for n in ("q", "k", "v", "g", "beta", "do")}
    o, S = gn.gnorm_delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], initial_state=x["S0"],
                              output_final_state=True)
    assert o.shape == y["v"].shape
    assert torch.equal(o.view_as(flat["o"]), flat["o"]) and torch.equal(S, flat["S"])
    grads = gn.gnorm_delta_bwd(y["do"], y["q"], y["k"], y["v"], y["g"], y["beta"],
                               initial_state=x["S0"], dfinal_state=x["dS"])
    for n, t in zip(GRADS, grads):
        assert torch.equal(t.view_as(flat[n]), flat[n]), n


def test_slices_of_one_projection():
    """q, k, v as columns of one wider tensor, g and beta of another."""
    x = make([150], 2, 4, 128, 64, state=True)
    ref = call(x)
    wide = torch.full((150, 2 * 256 + 256 + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    y = dict(x)
    for n, at, w in (("q", 0, 256), ("k", 256, 256), ("v", 512, 256)):
        wide[:, at:at + w] = x[n].reshape(150, w)
        y[n] = wide[:, at:at + w].unflatten(1, x[n].shape[1:])
    narrow = torch.zeros(150, 11, device="cuda")
    narrow[:, 1:5], narrow[:, 6:10] = x["g"], x["beta"]
    y["g"], y["beta"] = narrow[:, 1:5], narrow[:, 6:10]
    for n, t in call(y).items():
        assert torch.equal(t, ref[n]), n
    grad = torch.full_like(wide, 9.0)
    out = {"d" + n: grad[:, at:at + 256].unflatten(1, x[n].shape[1:])
           for n, at in (("q", 0), ("k", 256), ("v", 512))}
    out["dg"], out["dbeta"] = torch.empty_like(x["g"]), torch.empty_like(x["beta"])
    got = call(y, **out)
    for n in GRADS:
        assert torch.equal(got[n], ref[n]), n
    assert bool((grad[:, 768:] == 9.0).all())


def test_offsets_past_32_bits():
    T, ld = 130, 1 << 25
    x = make([T], 1, 1, 64, 64)
    ref = call(x)
    y = dict(x)
    for n in ("q", "v"):
        big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
        y[n] = big.as_strided((T, 1, 64), (ld, 64, 1))
        y[n].copy_(x[n])
    for n, t in call(y).items():
        if t is not None:
            assert torch.equal(t, ref[n]), n


def test_no_tokens():
    x = make([0, 0], 1, 2, 128, 64, state=True)
    got = call(x)
    assert torch.equal(got["S"], x["S0"]) and torch.equal(got["dS0"], x["dS"])
    assert got["o"].shape == (0, 2, 64)
    _, S = gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], cu_seqlens=x["cu"],
                              output_final_state=True)
    assert not S.any()


def test_bitwise_from_run_to_run():
    x = make([300, 41], 2, 4, 128, 128, state=True)
    first = call(x)
    for _ in range(3):
        for n, t in call(x).items():
            assert torch.equal(t, first[n]), n


def test_a_sequence_does_not_depend_on_its_neighbours():
    x = make([300, 41], 1, 2, 128, 128, state=True)
    both = call(x)
    y = {n: (t[300:] if torch.is_tensor(t) and n not in ("S0", "dS", "cu") else t)
         for n, t in x.items()}
    y["S0"], y["dS"] = x["S0"][1:], x["dS"][1:]
    y["cu"] = torch.tensor([0, 41], dtype=torch.int32, device="cuda")
    for n, t in call(y).items():
        want = both[n][1:] if n in ("S", "dS0") else both[n][300:]
        assert torch.equal(t, want), n


def test_states_carry_a_sequence_across_calls():
    x = make([192], 2, 2, 128, 128, state=True)
    o, S = gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                              initial_state=x["S0"], output_final_state=True)
    S1, parts = x["S0"], []
    for a, b in ((0, 64), (64, 128), (128, 192)):
        p, S1 = gn.gnorm_delta_fwd(*(x[n][a:b] for n in ("q", "k", "v", "g", "beta")),
                                   scale=x["scale"], initial_state=S1, output_final_state=True)
        parts.append(p)
    assert torch.equal(torch.cat(parts), o) and torch.equal(S1, S)


def test_autograd():
    x = make([80, 33], 2, 4, 64, 64, state=True)
    want = call(x)
    names = ("q", "k", "v", "g", "beta", "S0")
    leaf = {n: x[n].clone().requires_grad_() for n in names}
    o, S = gn.gated_delta_rule(leaf["q"], leaf["k"], leaf["v"], leaf["g"], leaf["beta"],
                               scale=x["scale"], cu_seqlens=x["cu"], initial_state=leaf["S0"])
    torch.autograd.backward([o, S], [x["do"], x["dS"]])
    assert torch.equal(o, want["o"]) and torch.equal(S, want["S"])
    for n in names:
        assert torch.equal(leaf[n].grad, want["d" + n]), n
    # one of the two outputs used, and an expanded gradient
    for pick in (0, 1):
        v = x["v"].clone().requires_grad_()
        out = gn.gated_delta_rule(x["q"], x["k"], v, x["g"], x["beta"], cu_seqlens=x["cu"])
        out[pick].sum().backward()
        y = dict(x, S0=None, do=torch.ones_like(x["do"]) * (1 - pick),
                 dS=torch.ones_like(x["dS"]) if pick else None)
        close(v.grad, recurrence(y)["dv"], "dv")


@pytest.mark.parametrize("V", [64, 128])
def test_thousands_of_sequences(V):
    """Sequences of 0 to 2 tokens: 3000 of them, as strips (V = 64) and as whole heads."""
    lens = [(1, 2, 0, 1)[(i * 7) % 4] for i in range(3000)]
    x = make(lens, 1, 1, 64, V, state=True, tail=3)
    got = call(x)
    n = sum(lens)
    # by hand: a token's step from its sequence's state, all first tokens, then all second ones
    cu = x["cu"].long()
    S = x["S0"].double()[:, 0]
    for i in range(2):
        at = (cu[1:] - cu[:-1] > i).nonzero()[:, 0]
        t = cu[at] + i
        q, k, v = (x[m][t, 0].double() for m in ("q", "k", "v"))
        R = x["g"][t, 0].double().exp()[:, None, None] * S[at]
        u = x["beta"][t].double() * (v - (k[:, :, None] * R).sum(1))
        R = R + k[:, :, None] * u[:, None, :]
        o = x["scale"] * (q[:, :, None] * R).sum(1)
        terms = x["scale"] * (q[:, :, None] * R).square().sum(1).sqrt()
        close(got["o"][t, 0], o, "o", size={"o": terms})
        S[at] = R
    close(got["S"], S[:, None], "S")
    assert not got["o"][n:].any()
    empty = (cu[1:] == cu[:-1]).nonzero()[:, 0]
    assert torch.equal(got["S"][empty], x["S0"][empty])
    assert torch.equal(got["dS0"][empty], x["dS"][empty])


def test_streams_and_workspaces_of_the_caller():
    """An explicit stream for every call, one workspace for calls in a row on it, and outputs of
    the caller's."""
    x = make([100, 60], 1, 2, 128, 128, state=True)
    want = call(x)
    s = torch.cuda.Stream()
    ws = torch.empty(gn.gnorm_delta_workspace_bytes(160, 2, 2, 128, 128, True), dtype=torch.uint8,
                     device="cuda")
    a = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    kw = dict(scale=x["scale"], cu_seqlens=x["cu"], initial_state=x["S0"], workspace_buf=ws, stream=s)
    out = {n: torch.empty_like(want[n]) for n in GRADS}
    o, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    torch.cuda.synchronize()
    for _ in range(2):
        r = gn.gnorm_delta_fwd(*a, o=o, final_state=S, **kw)
        assert r[0] is o and r[1].data_ptr() == S.data_ptr()
        r = gn.gnorm_delta_bwd(x["do"], *a, dfinal_state=x["dS"],
                               **{("dinitial_state" if n == "dS0" else n): t for n, t in out.items()}, **kw)
    s.synchronize()
    assert torch.equal(o, want["o"]) and torch.equal(S, want["S"])
    for n in GRADS:
        assert torch.equal(out[n], want[n]), n
    y = step_case(3, 1, 2, 128, 128, 5)
    ref = y["pool"].clone()
    o1 = step(y, ref, slots=y["slots"])
    pool = y["pool"].clone()
    torch.cuda.synchronize()
    o2 = step(y, pool, slots=y["slots"], stream=s)
    s.synchronize()
    assert torch.equal(o1, o2) and torch.equal(ref, pool)


def test_first_call_of_a_thread():
    """A thread that has made no CUDA call yet: both directions run there."""
    import threading

    x = make([70], 1, 2, 64, 64, state=True)
    want = call(x)
    torch.cuda.synchronize()
    for fn in (lambda: gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"],
                                          initial_state=x["S0"])[:1],
               lambda: gn.gnorm_delta_bwd(x["do"], x["q"], x["k"], x["v"], x["g"], x["beta"],
                                          initial_state=x["S0"], dfinal_state=x["dS"])):
        out = []
        t = threading.Thread(target=lambda: out.append(fn()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert len(out) == 1
        names = ("o",) if len(out[0]) == 1 else GRADS
        for n, got in zip(names, out[0]):
            assert torch.equal(got, want[n]), n


def test_gradients_against_differences():
    """The adjoint that the tests compare with, against central differences in FP64."""
    x = make([70], 1, 2, 64, 64, state=True)
    ref = recurrence(x)
    step = 1e-6
    for n, i in (("q", (40, 0, 3)), ("k", (20, 0, 60)), ("v", (5, 1, 9)), ("g", (33, 1)),
                 ("beta", (66, 0)), ("S0", (0, 1, 2, 3))):
        vals = []
        for sign in (1, -1):
            y = {m: (t.double().clone() if torch.is_tensor(t) and t.is_floating_point() else t)
                 for m, t in x.items()}
            y[n][i] += sign * step
            out = recurrence(y, grads=False)
            vals.append(float((out["o"] * x["do"].double()).sum() +
                              (out["S"] * x["dS"].double()).sum()))
        diff, want = (vals[0] - vals[1]) / (2 * step), float(ref["d" + n][i])
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want)), n


def test_delta_then_gated_norm():
    """The module: the rule, the gated norm of each head's output, and one backward through
    both; its step continues from the sequence's state."""
    x = make([90, 40], 2, 4, 128, 128, state=True)
    gen = torch.Generator(device="cuda").manual_seed(5)
    gate = torch.randn(x["v"].shape, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(x["v"].shape, generator=gen, device="cuda").bfloat16()
    mod = gn.GatedDeltaNorm(128, dtype=torch.float32, device="cuda")
    v = x["v"].clone().requires_grad_()
    y, S = mod(x["q"], x["k"], v, x["g"], x["beta"], gate, scale=x["scale"], cu_seqlens=x["cu"],
               initial_state=x["S0"])
    y.backward(dy)
    o, S2 = gn.gnorm_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                               cu_seqlens=x["cu"], initial_state=x["S0"], output_final_state=True)
    w = mod.weight.detach()
    y2, rstd = gn.gnorm_fwd(o, gate, w, mod.eps)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    do, _, dw = gn.gnorm_bwd(dy, o, gate, w, rstd, dw_fp32=True)
    assert torch.equal(mod.weight.grad, dw)
    dv = gn.gnorm_delta_bwd(do, x["q"], x["k"], x["v"], x["g"], x["beta"], scale=x["scale"],
                            cu_seqlens=x["cu"], initial_state=x["S0"])[2]
    assert torch.equal(v.grad, dv)
    # a step of both sequences, then the same tokens appended to them
    z = make([1, 1], 2, 4, 128, 128, seed=9)
    state = S.detach().clone()
    y1 = mod.step(z["q"], z["k"], z["v"], z["g"], z["beta"], gate[:2], state, scale=x["scale"])
    ref = recurrence(dict(z, S0=S.detach(), dS=None), grads=False)
    close(state, ref["S"], "S", 1e-5)
    o1 = ref["o"]
    sg = gate[:2].double()
    want = o1 * (o1.square().mean(-1, keepdim=True) + mod.eps).rsqrt() * sg * torch.sigmoid(sg)
    # the norm's input is BF16 here: half a step of o goes through the norm
    err = (y1.double() - want).abs()
    rms = want.square().mean(-1, keepdim=True).sqrt()
    assert bool((err <= 3 * 2.0 ** -8 * torch.maximum(rms, want.abs()) + 1e-4).all())


def test_captured_and_replayed():
    x = make([120, 75], 1, 2, 128, 128, state=True)
    eager = call(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for _ in range(2):  # two graphs, replayed in turn, each with a workspace of its own
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(call(x))
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for n, t in out.items():
            assert torch.equal(t, eager[n]), n


def test_on_another_stream():
    x = make([500], 2, 4, 128, 128, state=True)
    want = call(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = call(x)
    here = call(x)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.equal(here[n], want[n]), n


# ------------------------------------------------------------------------------ the step

def step_case(B, Hk, Hv, K, V, pool, beta=torch.float32, seed=0):
    x = make([1] * B, Hk, Hv, K, V, beta=beta, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x["pool"] = 0.3 * torch.randn(pool, Hv, K, V, generator=gen, device="cuda")
    x["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:B].to(torch.int32)
    return x


def step(x, state, **kw):
    return gn.gnorm_delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state,
                               scale=x["scale"], **kw)


@pytest.mark.parametrize("K,V,Hk,Hv", HEADS)
@pytest.mark.parametrize("B", [1, 3, 40, 130])
def test_step(B, K, V, Hk, Hv):
    x = step_case(B, Hk, Hv, K, V, B + 7, torch.bfloat16 if B % 2 else torch.float32)
    state = x["pool"].clone()
    o = step(x, state, slots=x["slots"])
    at = x["slots"].long()
    ref = recurrence(dict(x, S0=x["pool"][at]), grads=False)
    close(o, ref["o"], "o", 1e-5)
    close(state[at], ref["S"], "S", 1e-5)
    rest = torch.ones(B + 7, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(state[rest], x["pool"][rest])


def test_step_padding_rows():
    x = step_case(6, 1, 2, 128, 128, 9)
    want = x["pool"].clone()
    o_all = step(x, want, slots=x["slots"])
    slots = x["slots"].clone()
    slots[1], slots[4] = -1, 9
    for n in ("q", "k", "v", "g", "beta"):
        x[n][[1, 4]] = float("nan")
    state = x["pool"].clone()
    o = torch.full_like(x["v"], 7.0)
    step(x, state, slots=slots, o=o)
    live = [0, 2, 3, 5]
    assert not o[[1, 4]].any() and torch.equal(o[live], o_all[live])
    at = x["slots"].long()
    assert torch.equal(state[at[live]], want[at[live]])
    assert torch.equal(state[at[[1, 4]]], x["pool"][at[[1, 4]]])


@pytest.mark.parametrize("B", [7, 300])
def test_step_rows_that_share_a_slot(B):
    """Consecutive tokens of one sequence in one call."""
    x = step_case(B, 1, 2, 128, 64, 3)
    slots = torch.randint(-1, 3, (B,), device="cuda", dtype=torch.int32,
                          generator=torch.Generator(device="cuda").manual_seed(2))
    state = x["pool"].clone()
    o = step(x, state, slots=slots)
    for s in range(3):
        at = (slots == s).nonzero()[:, 0]
        y = {n: (t[at] if torch.is_tensor(t) and n in ("q", "k", "v", "g", "beta") else t)
             for n, t in x.items()}
        ref = recurrence(dict(y, lens=[at.numel()], S0=x["pool"][s:s + 1]), grads=False)
        close(o[at], ref["o"], "o", 1e-5)
        close(state[s:s + 1], ref["S"], "S", 1e-5)
    assert not o[slots < 0].any()


def test_step_without_slots_and_a_strided_pool():
    x = step_case(5, 2, 4, 128, 128, 8)
    want = x["pool"].clone()
    o1 = step(x, want, slots=torch.arange(5, device="cuda", dtype=torch.int32))
    state = x["pool"].clone()
    assert torch.equal(step(x, state), o1) and torch.equal(state, want)
    n = 4 * 128 * 128
    wide = torch.full((8, n + 64), 5.0, device="cuda")
    wide[:, :n] = x["pool"].view(8, n)
    pool = wide[:, :n].unflatten(1, (4, 128, 128))
    assert torch.equal(step(x, pool), o1) and torch.equal(pool, want)
    assert bool((wide[:, n:] == 5.0).all())


def test_step_pool_past_32_bits():
    x = step_case(2, 1, 1, 128, 128, 2)
    far = torch.empty(1 << 34, dtype=torch.uint8, device="cuda").view(torch.float32)
    pool = far.as_strided((2, 1, 128, 128), ((1 << 32) - 128 * 128, 128 * 128, 128, 1))
    pool.copy_(x["pool"])
    want = x["pool"].clone()
    o = step(x, want)
    assert torch.equal(step(x, pool), o) and torch.equal(pool, want)


def test_step_equals_the_sequence():
    """T steps and one call over T tokens, from the same state."""
    T = 100
    x = make([T], 2, 4, 128, 128, state=True)
    seq = call(x)
    state = x["S0"].clone()
    for t in range(T):
        y = {n: x[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")}
        o = gn.gnorm_delta_step(y["q"], y["k"], y["v"], y["g"], y["beta"], state)
        close(o, seq["o"][t:t + 1].double(), "o", SPLIT + 2.0 ** -8)
    close(state, seq["S"].double(), "S")


def test_step_resets_and_replays():
    x = step_case(4, 1, 2, 64, 64, 4)
    x["g"][2] = float("-inf")
    state = x["pool"].clone()
    o = step(x, state)
    ref = recurrence(dict(x, g=x["g"].clamp(min=-700.0), S0=x["pool"]), grads=False)
    close(o, ref["o"], "o", 1e-5)
    close(state, ref["S"], "S", 1e-5)
    pool = x["pool"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o2 = step(x, pool)
    torch.cuda.current_stream().wait_stream(s)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, o) and torch.equal(pool, state)


# ------------------------------------------------------------------------------ refusals

def test_refusals():
    x = make([64], 2, 4, 64, 64, state=True)
    a = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    with pytest.raises(gn.GnormError):  # o over v
        gn.gnorm_delta_fwd(*a, o=x["v"])
    with pytest.raises(gn.GnormError):  # the final state over the initial one
        gn.gnorm_delta_fwd(*a, initial_state=x["S0"], final_state=x["S0"])
    with pytest.raises(gn.GnormError):
        gn.gnorm_delta_fwd(*a, scale=float("inf"))
    with pytest.raises(gn.GnormError):  # a head size that no kernel has
        gn.gnorm_delta_fwd(x["q"][..., :32].contiguous(), x["k"][..., :32].contiguous(), *a[2:])
    with pytest.raises(gn.GnormError):  # 4 value heads over 3 key heads
        gn.gnorm_delta_fwd(*(t.repeat(1, 2, 1)[:, :3].contiguous() for t in a[:2]), *a[2:])
    with pytest.raises(gn.GnormError):  # an odd token stride
        wide = torch.zeros(64, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        gn.gnorm_delta_fwd(*a[:2], wide[:, :256].unflatten(1, (4, 64)), *a[3:])
    with pytest.raises(gn.GnormError):
        gn.gnorm_delta_bwd(x["do"], *a, workspace_buf=torch.empty(256, dtype=torch.uint8,
                                                                  device="cuda"))
    with pytest.raises(TypeError):
        gn.gnorm_delta_fwd(x["q"].float(), *a[1:])
    with pytest.raises(TypeError):
        gn.gnorm_delta_fwd(*a[:3], x["g"].bfloat16(), x["beta"])
    with pytest.raises(TypeError):
        gn.gnorm_delta_fwd(*a, cu_seqlens=x["cu"].long())
    with pytest.raises(ValueError):
        gn.gnorm_delta_fwd(*a, cu_seqlens=x["cu"].cpu())
    with pytest.raises(ValueError):  # heads not packed within a token
        gn.gnorm_delta_fwd(x["q"].transpose(0, 1).contiguous().transpose(0, 1), *a[1:])
    with pytest.raises(ValueError):
        gn.gnorm_delta_fwd(*a, initial_state=x["S0"][:, :2])
    with pytest.raises(ValueError):  # fewer tokens in one of them
        gn.gnorm_delta_fwd(x["q"], x["k"][:32], *a[2:])
    with pytest.raises(ValueError):
        gn.gnorm_delta_bwd(x["do"], *a, cu_seqlens=x["cu"], dq=torch.empty_like(x["q"]))
    pool = torch.zeros(3, 4, 64, 64, device="cuda")
    y = tuple(t[:5] for t in a)
    with pytest.raises(gn.GnormError):  # more rows than slots
        gn.gnorm_delta_step(*y, pool)
    with pytest.raises(TypeError):
        gn.gnorm_delta_step(*y, pool, slots=torch.zeros(5, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gn.gnorm_delta_step(*y, pool, slots=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gn.gnorm_delta_step(*y, pool.transpose(2, 3))
    with pytest.raises(TypeError):
        gn.gnorm_delta_step(*y, pool.bfloat16())
