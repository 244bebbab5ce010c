"""The block norm (gnorm_block_fwd / gnorm_block_bwd) against its formulas in FP64 (GPU).

Tolerances, from the arithmetic: an FP32 path of about 20 operations and row sums of at most
16384 terms in tree order is within 1e-5 of the exact value relative to the row's RMS (each
operation is off by at most 2^-24 relative, the MUFU exp2 and reciprocal by a few of those);
an output in BF16 adds half a step, 2^-8 relative.  Sums over rows (dw1, dw2, dalpha) are FP32
sums of M terms whose error grows as a random walk, checked relative to the sums' RMS.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn

EPS = 1e-6


def make(M, N, *, gate, res, wt=torch.float32, seed=0, dh=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    return dict(a=rand(M, N).bfloat16(), r=(2 * rand(M, N)).to(res),
                g=(2 * rand(M, N)).bfloat16() if gate else None,
                w1=(1 + 0.1 * rand(N)).to(wt), w2=(1 + 0.1 * rand(N)).to(wt),
                alpha=torch.full((1,), 0.7, device="cuda"),
                dh=rand(M, N).to(res) if dh else None, dz=rand(M, N).bfloat16())


def reference(x, eps1=EPS, eps2=EPS):
    d = {n: None if t is None else t.double() for n, t in x.items()}
    N = d["a"].shape[-1]
    alpha = d["alpha"] if d["alpha"] is not None else torch.ones(1, device="cuda").double()
    r1 = (d["a"].square().mean(-1, keepdim=True) + eps1).rsqrt()
    ah = d["a"] * r1
    b = ah * d["w1"]
    sg = torch.sigmoid(d["g"]) if d["g"] is not None else None
    s = d["g"] * sg if sg is not None else torch.ones_like(b)
    h = d["r"] + alpha * s * b
    r2 = (h.square().mean(-1, keepdim=True) + eps2).rsqrt()
    hh = h * r2
    u2 = d["dz"] * d["w2"]
    dr = r2 * (u2 - hh * (u2 * hh).sum(-1, keepdim=True) / N)
    if d["dh"] is not None:
        dr = dr + d["dh"]
    t = dr * s
    u1 = alpha * t * d["w1"]
    out = dict(h=h, z=hh * d["w2"], rstd1=r1[:, 0], rstd2=r2[:, 0], dr=dr,
               da=r1 * (u1 - ah * (u1 * ah).sum(-1, keepdim=True) / N),
               dw1=alpha * (t * ah).sum(0), dw2=(d["dz"] * hh).sum(0),
               dalpha=(t * b).sum().reshape(1))
    if sg is not None:
        out["dg"] = alpha * dr * b * sg * (1 + d["g"] * (1 - sg))
    return out


def close(got, ref, name, f32=1e-5):
    assert got.shape == ref.shape, name
    err = (got.double() - ref).abs()
    rms = ref.square().mean(-1, keepdim=True).sqrt() if ref.dim() > 1 else \
        ref.square().mean().sqrt()
    half = torch.finfo(got.dtype).eps / 2 if got.dtype == torch.bfloat16 else 0.0
    tol = half * ref.abs() + f32 * torch.maximum(rms, ref.abs()) + 1e-30
    assert bool((err <= tol).all()), (name, float((err / tol).max()))


def check(x, M, N, **kw):
    alpha, g = x["alpha"], x["g"]
    h, z, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=g, alpha=alpha)
    out = gn.gnorm_block_bwd(x["dh"], x["dz"], x["a"], x["r"], x["w1"], x["w2"], r1, r2, g=g,
                             alpha=alpha, dw_fp32=True, **kw)
    ref = reference(x)
    for t, n in ((h, "h"), (z, "z"), (r1, "rstd1"), (r2, "rstd2")):
        close(t, ref[n], n)
    for t, n in zip(out, ("da", "dr", "dg", "dw1", "dw2")):
        if t is not None:
            close(t, ref[n], n, 2e-5)
    assert (out[2] is None) == (g is None)
    if alpha is not None:
        # a sum of M N terms: its error is a random walk of their roundings
        rms = float((ref["dr"].square().mean() * M * N).sqrt())
        assert abs(float(out[5]) - float(ref["dalpha"])) <= 1e-5 * (abs(float(ref["dalpha"])) + rms)
    else:
        assert out[5] is None
    assert gn.gnorm_device_error(reset=True) == 0
    return (h, z, r1, r2) + out


SHAPES = [(1, 8), (3, 64), (257, 72), (1, 128), (1031, 128), (4099, 248), (65, 512), (33, 1000),
          (2051, 1024), (147, 2040), (149, 4096), (700, 4096), (19, 5120), (31, 8192),
          (5, 12288), (3, 16384)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("gate", [True, False])
def test_bf16_residual(M, N, gate):
    check(make(M, N, gate=gate, res=torch.bfloat16, seed=M + N), M, N)


@pytest.mark.parametrize("M,N", [s for s in SHAPES if s[1] < 16384])
def test_fp32_residual(M, N):
    check(make(M, N, gate=True, res=torch.float32, wt=torch.bfloat16, seed=M), M, N)


@pytest.mark.parametrize("M,N", [(301, 256), (37, 4096)])
def test_no_dh_no_alpha(M, N):
    x = make(M, N, gate=True, res=torch.bfloat16, dh=False)
    x["alpha"] = None
    check(x, M, N)


def test_many_rows():
    check(make(262144, 128, gate=True, res=torch.bfloat16), 262144, 128)


def test_alpha_zero_keeps_its_gradient():
    """A residual scale that starts at zero still gets a gradient (ReZero), and the branch
    none."""
    M, N = 129, 512
    x = make(M, N, gate=True, res=torch.bfloat16)
    x["alpha"] = torch.zeros(1, device="cuda")
    out = check(x, M, N)
    assert torch.equal(out[0], x["r"]) and float(out[9]) != 0.0
    assert not out[4].any() and not out[6].any() and not out[7].any()


def test_bf16_weight_gradients():
    M, N = 513, 1024
    x = make(M, N, gate=True, res=torch.bfloat16, wt=torch.bfloat16)
    _, _, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=x["g"],
                                      alpha=x["alpha"])
    out = gn.gnorm_block_bwd(x["dh"], x["dz"], x["a"], x["r"], x["w1"], x["w2"], r1, r2,
                             g=x["g"], alpha=x["alpha"])
    ref = reference(x)
    assert out[3].dtype == out[4].dtype == torch.bfloat16
    close(out[3], ref["dw1"], "dw1", 2e-5)
    close(out[4], ref["dw2"], "dw2", 2e-5)


@pytest.mark.parametrize("M,N", [(300, 256), (70, 4096)])
def test_strided_rows_leave_the_padding(M, N):
    x = make(M, N, gate=True, res=torch.bfloat16)
    ref = check(x, M, N)
    buf = torch.full((M, 2 * N + 16), -7.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :N], buf[:, N:2 * N] = x["a"], x["g"]
    y = dict(x, a=buf[:, :N], g=buf[:, N:2 * N])
    grad = torch.full((M, 2 * N + 16), -7.0, dtype=torch.bfloat16, device="cuda")
    got = check(y, M, N, da=grad[:, :N], dg=grad[:, N:2 * N])
    for p, q in zip(ref, got):
        assert torch.equal(p, q)
    assert bool((buf[:, 2 * N:] == -7).all()) and bool((grad[:, 2 * N:] == -7).all())


def test_bitwise_from_run_to_run():
    M, N = 9001, 512
    x = make(M, N, gate=True, res=torch.bfloat16)
    first = check(x, M, N)
    for _ in range(3):
        for p, q in zip(first, check(x, M, N)):
            assert torch.equal(p, q)


def test_non_finite_rows_stay_in_their_rows():
    M, N = 40, 1024
    x = make(M, N, gate=True, res=torch.bfloat16)
    clean = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=x["g"], alpha=x["alpha"])
    x["a"][3, 5] = float("nan")
    x["r"][7, 0] = float("inf")
    x["g"][11, 9] = float("-inf")
    h, z, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=x["g"],
                                      alpha=x["alpha"])
    ref = reference(x)
    for t, n in ((h, "h"), (z, "z")):
        assert torch.equal(torch.isnan(t), torch.isnan(ref[n]))
    keep = [i for i in range(M) if i not in (3, 7, 11)]
    for t, c in ((h, clean[0]), (z, clean[1])):
        assert torch.equal(t[keep], c[keep])


def test_empty_batch():
    N = 256
    x = make(0, N, gate=True, res=torch.bfloat16)
    h, z, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=x["g"],
                                      alpha=x["alpha"])
    assert h.shape == z.shape == (0, N) and r1.numel() == 0
    out = gn.gnorm_block_bwd(x["dh"], x["dz"], x["a"], x["r"], x["w1"], x["w2"], r1, r2,
                             g=x["g"], alpha=x["alpha"], dw_fp32=True)
    assert not out[3].any() and not out[4].any() and not out[5].any()


def test_autograd_equals_the_calls_and_finite_differences():
    M, N = 6, 64
    x = make(M, N, gate=True, res=torch.float32)
    mod = gn.BlockRMSNorm(N, alpha=0.7, dtype=torch.float32, device="cuda")
    with torch.no_grad():
        mod.weight_post.copy_(x["w1"])
        mod.weight_pre.copy_(x["w2"])
    a, r, g = (x[n].clone().requires_grad_() for n in ("a", "r", "g"))
    h, z = mod(a, r, g)
    torch.autograd.backward([h, z], [x["dh"], x["dz"]])
    h2, z2, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=x["g"],
                                        alpha=mod.alpha.detach())
    out = gn.gnorm_block_bwd(x["dh"], x["dz"], x["a"], x["r"], x["w1"], x["w2"], r1, r2,
                             g=x["g"], alpha=mod.alpha.detach(), dw_fp32=True)
    assert torch.equal(h, h2) and torch.equal(z, z2)
    for p, q in zip((a.grad, r.grad, g.grad, mod.weight_post.grad, mod.weight_pre.grad,
                     mod.alpha.grad), out):
        assert torch.equal(p, q)
    # the formula's gradient against central differences, in FP64
    step = 1e-6
    for n, i in (("r", (2, 3)), ("a", (1, 5)), ("g", (4, 60)), ("w1", (7,)), ("alpha", (0,))):
        vals = []
        for sgn in (1, -1):
            y = {k: None if t is None else t.double().clone() for k, t in x.items()}
            y[n][i] += sgn * step
            o = reference(y)
            vals.append(float((o["h"] * x["dh"].double()).sum() + (o["z"] * x["dz"].double()).sum()))
        diff = (vals[0] - vals[1]) / (2 * step)
        want = float(reference(x)[{"w1": "dw1", "alpha": "dalpha"}.get(n, "d" + n)][i])
        assert abs(diff - want) <= 1e-5 * max(1.0, abs(want)), n


def test_only_z_used():
    M, N = 50, 256
    x = make(M, N, gate=False, res=torch.bfloat16)
    a = x["a"].clone().requires_grad_()
    _, z = gn.block_rmsnorm(a, x["r"], x["w1"], x["w2"])
    z.backward(x["dz"])
    ref = reference(dict(x, dh=None, alpha=None))
    close(a.grad, ref["da"], "da", 2e-5)


def test_captured_and_replayed():
    M, N = 600, 512
    x = make(M, N, gate=True, res=torch.bfloat16)
    eager = check(x, M, N)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            h, z, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], EPS, g=x["g"],
                                              alpha=x["alpha"])
            out = gn.gnorm_block_bwd(x["dh"], x["dz"], x["a"], x["r"], x["w1"], x["w2"], r1, r2,
                                     g=x["g"], alpha=x["alpha"], dw_fp32=True)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for p, q in zip(eager, (h, z, r1, r2) + out):
        assert torch.equal(p, q)


def test_refusals():
    x = make(16, 256, gate=True, res=torch.bfloat16)
    args = (x["a"], x["r"], x["w1"], x["w2"])
    with pytest.raises(gn.GnormError):  # h over r
        gn.gnorm_block_fwd(*args, EPS, g=x["g"], h=x["r"])
    with pytest.raises(gn.GnormError):
        gn.gnorm_block_fwd(*args, -1.0)
    with pytest.raises(TypeError):
        gn.gnorm_block_fwd(x["a"].float(), x["r"], x["w1"], x["w2"])
    with pytest.raises(TypeError):  # weights of two types
        gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"].bfloat16())
    with pytest.raises(ValueError):
        gn.gnorm_block_fwd(x["a"], x["r"][:8], x["w1"], x["w2"])
    with pytest.raises(ValueError):
        gn.gnorm_block_fwd(x["a"], x["r"], x["w1"].cpu(), x["w2"])
    _, _, r1, r2 = gn.gnorm_block_fwd(*args, EPS, g=x["g"])
    with pytest.raises(gn.GnormError):  # a workspace too small
        gn.gnorm_block_bwd(x["dh"], x["dz"], *args, r1, r2, g=x["g"],
                           workspace_buf=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gn.gnorm_block_bwd(x["dh"], x["dz"], *args, r1, r2, dg=x["g"].clone())
