"""The operators of a linear-attention block around the gated norm, as cases to be timed.

Two operators, each in the forms in which a program calls it:

``block``: the norm after a block, its gate, the residual scale and the norm before the next
block, in one pass.  With rows a (the block's output), r (the residual), an optional gate g,
a residual scale alpha (one FP32 value on the device) and weights w1, w2::

    b = a * rsqrt(mean(a^2) + eps) * w1
    h = r + alpha * silu(g) * b          (silu(g) = 1 where there is no gate)
    z = h * rsqrt(mean(h^2) + eps) * w2

``delta``: the gated delta rule, per sequence and value head, S of K x V values::

    S_t = exp(g_t) S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t)
    o_t = scale * S_t^T q_t

over packed sequences (forward; forward and gradients), and for one token of each sequence
with the states kept in a pool.

``own`` says whether ``run`` computes the plain form or calls ``gated_norm_b200``.
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-6


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of a small batch: the residual update between two layers
        dict(name="block_fwd_16x4096", op="block", M=16, N=4096, gate=True, res="bf16",
             train=False),
        # the widest of the framework's workloads, its forward alone (evaluation, prefill)
        dict(name="block_fwd_16384x4096", op="block", M=16384, N=4096, gate=True, res="bf16",
             train=False),
        # a training micro-batch of a small model whose residual is kept in FP32, without a
        # gate, at an odd width and an odd number of rows
        dict(name="block_train_4099x1000", op="block", M=4099, N=1000, gate=False, res="fp32",
             train=True),
        # a training batch at the framework's widest workload
        dict(name="block_train_16384x4096", op="block", M=16384, N=4096, gate=True, res="bf16",
             train=True),
        # narrow rows, many of them (the framework's 262144 x 256 workload)
        dict(name="block_train_262144x256", op="block", M=262144, N=256, gate=True, res="bf16",
             train=True),
        # decoding for a handful of users: latency
        dict(name="delta_step_4", op="step", B=4, Hk=8, Hv=16, K=128, V=128, pool=8,
             beta="fp32"),
        # decoding for many users, states in a pool
        dict(name="delta_step_256", op="step", B=256, Hk=16, Hv=32, K=128, V=128, pool=320,
             beta="bf16"),
        # prefill of a few prompts of odd lengths, continuing from states
        dict(name="delta_fwd_5_prompts", op="delta", T=2777, B=5, Hk=8, Hv=16, K=128, V=128,
             state=True, beta="bf16", train=False),
        # prefill of one long prompt
        dict(name="delta_fwd_long", op="delta", T=16384, B=1, Hk=16, Hv=32, K=128, V=128,
             state=False, beta="fp32", train=False),
        # training on a few short documents with small heads
        dict(name="delta_train_64", op="delta", T=1531, B=3, Hk=6, Hv=6, K=64, V=64,
             state=False, beta="fp32", train=True),
        # training on packed documents, states carried in and out (the context is cut)
        dict(name="delta_train_packed", op="delta", T=4096, B=7, Hk=8, Hv=16, K=128, V=128,
             state=True, beta="fp32", train=True),
        # a training batch of one long context: the framework's 512 heads x 128 tokens as
        # 16 heads x 8192 tokens
        dict(name="delta_train_long", op="delta", T=8192, B=1, Hk=16, Hv=16, K=128, V=128,
             state=False, beta="bf16", train=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["block", "block", "step", "delta", "delta"])
    if op == "block":
        N = 8 * _log_int(rng, 8, 1024)
        M = _log_int(rng, 1, min(262144, (1 << 26) // N))
        return dict(op=op, M=M, N=N, gate=rng.random() < 0.7, res=rng.choice(["bf16", "fp32"])
                    if M * N <= 1 << 25 else "bf16", train=rng.random() < 0.6)
    K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    Hk = rng.choice([1, 2, 4, 6, 8, 16])
    Hv = Hk * rng.choice([1, 1, 2] if Hk > 4 else [1, 2, 4])
    beta = rng.choice(["fp32", "bf16"])
    if op == "step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, Hk=Hk, Hv=Hv, K=K, V=V, pool=B + rng.randrange(0, 64), beta=beta)
    train = rng.random() < 0.5
    T = _log_int(rng, 1, min(8192, 8192 * 16 // Hv) if train else 16384)
    B = min(T, rng.choice([1, 1, 2, 3, 5, 8]))
    return dict(op=op, T=T, B=B, Hk=Hk, Hv=Hv, K=K, V=V, state=rng.random() < 0.5, beta=beta,
                train=train)


# ----------------------------------------------------------------------------- the inputs

def _lengths(T, B, seed):
    """B sequence lengths >= 1 that sum to T, uneven."""
    g = torch.Generator().manual_seed(seed)
    if B == 1:
        return [T]
    cuts = sorted((torch.randperm(T - 1, generator=g)[:B - 1] + 1).tolist())
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = case

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(c)
    if c["op"] == "block":
        M, N = c["M"], c["N"]
        rt = torch.float32 if c["res"] == "fp32" else torch.bfloat16
        s["a"] = rand(M, N).bfloat16()
        s["r"] = (2.0 * rand(M, N)).to(rt)
        s["g"] = rand(M, N).bfloat16() if c["gate"] else None
        s["w1"] = 1.0 + 0.1 * rand(N)
        s["w2"] = 1.0 + 0.1 * rand(N)
        s["alpha"] = torch.full((1,), 0.5, device=dev)
        if c["train"]:
            # the upstream gradient has a part along the block's output, as it has while the
            # residual scale is still being learned
            along = s["a"].float() if s["g"] is None else s["a"].float() * s["g"].float()
            s["dh"] = (rand(M, N) + 0.1 * along).to(rt)
            s["dz"] = rand(M, N).bfloat16()
        return s

    T = c["B"] if c["op"] == "step" else c["T"]
    Hk, Hv, K, V = c["Hk"], c["Hv"], c["K"], c["V"]
    # keys and queries of unit length (keys of a head share a direction in part); decay rates
    # and step sizes as such layers are initialised: A in [1, 16] per head, dt in [1e-3, 0.1]
    q = torch.nn.functional.normalize(rand(T, Hk, K), dim=-1)
    k = torch.nn.functional.normalize(rand(T, Hk, K) + 0.5 * rand(1, Hk, K), dim=-1)
    s["q"], s["k"], s["v"] = q.bfloat16(), k.bfloat16(), rand(T, Hv, V).bfloat16()
    u = torch.rand(2, Hv, generator=gen, device=dev)
    rate, dt = 1.0 + 15.0 * u[0], torch.exp(math.log(1e-3) + u[1] * math.log(100.0))
    bias = dt + torch.log(-torch.expm1(-dt))
    s["gk"] = -rate * torch.nn.functional.softplus(0.5 * rand(T, Hv) + bias)
    s["beta"] = torch.sigmoid(rand(T, Hv)).to(
        torch.float32 if c["beta"] == "fp32" else torch.bfloat16)
    s["scale"] = K ** -0.5
    if c["op"] == "step":
        s["pool_state"] = 0.3 * rand(c["pool"], Hv, K, V)
        s["slots"] = torch.randperm(c["pool"], generator=gen, device=dev)[:T].to(torch.int32)
        return s
    lens = _lengths(T, c["B"], seed)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["max_len"] = max(lens)
    s["lens"] = lens
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["S0"] = 0.3 * rand(c["B"], Hv, K, V) if c["state"] else None
    if c["train"]:
        s["do"] = rand(T, Hv, V).bfloat16()
        s["dS"] = 0.1 * rand(c["B"], Hv, K, V) if c["state"] else None
    return s


def work(case):
    c = case
    if c["op"] == "block":
        M, N = c["M"], c["N"]
        e = 4 if c["res"] == "fp32" else 2
        g = 1 if c["gate"] else 0
        # forward: a, g, r in; h, z out
        nbytes = M * N * (2 + 2 * g + e + e + 2)
        flops = M * N * (12 + 5 * g)
        if c["train"]:
            # backward: dh and dz in; da, dg, dr out (a, g and r are read once for both)
            nbytes += M * N * (e + 2 + 2 + 2 * g + e) + 16 * N
            flops += M * N * (30 + 12 * g)
        return {"bytes": nbytes + 8 * N, "flops": flops}
    Hk, Hv, K, V = c["Hk"], c["Hv"], c["K"], c["V"]
    be = 4 if c["beta"] == "fp32" else 2
    T = c["B"] if c["op"] == "step" else c["T"]
    tok = 2 * (2 * Hk * K + Hv * V) + Hv * (4 + be)  # q, k, v, g, beta of one token
    if c["op"] == "step":
        return {"bytes": T * (tok + 2 * Hv * V + 8 * Hv * K * V), "flops": 7 * T * Hv * K * V}
    nbytes = T * (tok + 2 * Hv * V)
    nbytes += 4 * c["B"] * Hv * K * V * ((2 if c["state"] else 1) if not c["train"] else
                                         (4 if c["state"] else 0))
    # products of the recurrence by the token: S^T k, k u^T, S^T q, each 2 K V
    flops = 6 * T * Hv * K * V
    if c["train"]:
        # do in; dq, dk, dv, dg, dbeta out.  Gradients: twice the products of the forward
        nbytes += T * (2 * Hv * V + tok)
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------------ the plain forms

def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _block(a, r, g, alpha, w1, w2):
    b = _norm(a, w1)
    if g is not None:
        b = g * torch.sigmoid(g) * b
    h = r + alpha * b
    return h, _norm(h, w2)


def _plain_block(s):
    # leaves of their own: the inputs keep no history
    x = {n: None if s[n] is None else s[n].detach().float().requires_grad_(s["train"])
         for n in ("a", "r", "g", "alpha", "w1", "w2")}
    h, z = _block(x["a"], x["r"], x["g"], x["alpha"], x["w1"], x["w2"])
    out = {"h": h.detach().to(s["r"].dtype), "z": z.detach().bfloat16()}
    if s["train"]:
        names = [n for n in x if x[n] is not None]
        grads = torch.autograd.grad([h, z], [x[n] for n in names],
                                    [s["dh"].float(), s["dz"].float()])
        for n, d in zip(names, grads):
            out["d" + n] = d.to(s[n].dtype)
    return out


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower triangular A, by halves: T21 = -T22 A21 T11."""
    C = A.shape[-1]
    T = torch.eye(C, dtype=A.dtype, device=A.device).expand(A.shape)
    n = 1
    while n < C:
        m = C // (2 * n)
        blocks = T.reshape(*T.shape[:-2], m, 2 * n, m, 2 * n)
        ab = A.reshape(*A.shape[:-2], m, 2 * n, m, 2 * n)
        i = torch.arange(m, device=A.device)
        d = blocks.movedim(-2, -3)[..., i, i, :, :]
        da = ab.movedim(-2, -3)[..., i, i, :, :]
        t11, t22 = d[..., :n, :n], d[..., n:, n:]
        t21 = -t22 @ da[..., n:, :n] @ t11
        top = torch.cat([t11, torch.zeros_like(t21)], -1)
        d = torch.cat([top, torch.cat([t21, t22], -1)], -2)
        eye = torch.eye(m, dtype=A.dtype, device=A.device)[:, None, :, None]
        T = (d[..., :, :, None, :] * eye).reshape(A.shape)
        n *= 2
    return T


def _plain_delta_forward(q, k, v, g, beta, S0, s):
    """o and the final states, in FP32, chunk by chunk.  The loop goes over the chunks: each
    needs the state that the one before leaves."""
    T, Hk, K = q.shape
    Hv, V = v.shape[1:]
    B, dev = s["cu"].numel() - 1, q.device
    n = -(-s["max_len"] // CHUNK)
    L = n * CHUNK
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(L, device=dev)
    live = at < cu[1:, None]
    at = at.clamp(max=T - 1)

    def lay(x):  # [T, H, D] -> [B, H, n, C, D], zero behind each sequence
        y = x[at] * live[..., None, None]
        y = y.reshape(B, n, CHUNK, x.shape[1], x.shape[2]).permute(0, 3, 1, 2, 4)
        return y.repeat_interleave(Hv // x.shape[1], 1) if x.shape[1] != Hv else y

    Q, Kx, Vx = lay(q), lay(k), lay(v)
    G = lay(g[..., None])[..., 0].double().cumsum(-1)
    Bt = lay(beta[..., None])
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    into = torch.exp(G).float()[..., None]
    left = torch.exp(G[..., -1:] - G).float()[..., None]
    whole = torch.exp(G[..., -1]).float()[..., None, None]
    A = Bt * (Kx @ Kx.transpose(-1, -2)) * (D * low.tril(-1))
    Ti = _unit_lower_inverse(A)
    P = (Q @ Kx.transpose(-1, -2)) * D
    kin, qin, kout = Kx * into, Q * into, (Kx * left).transpose(-1, -2)
    S = torch.zeros(B, Hv, K, V, device=dev) if S0 is None else S0
    outs = []
    for c in range(n):
        U = Ti[:, :, c] @ (Bt[:, :, c] * (Vx[:, :, c] - kin[:, :, c] @ S))
        outs.append(qin[:, :, c] @ S + P[:, :, c] @ U)
        S = whole[:, :, c] * S + kout[:, :, c] @ U
    o = s["scale"] * torch.stack(outs, 2).permute(0, 2, 3, 1, 4).reshape(B * L, Hv, V)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b * L + t - cu[b]], S


def _plain_delta(s):
    names = ["q", "k", "v", "gk", "beta"] + (["S0"] if s["S0"] is not None else [])
    x = {n: s[n].detach().float().requires_grad_(s["train"]) for n in names}
    o, S = _plain_delta_forward(x["q"], x["k"], x["v"], x["gk"], x["beta"], x.get("S0"), s)
    out = {"o": o.detach().bfloat16()}
    if not s["train"] or s["S0"] is not None:
        out["state"] = S.detach()
    if s["train"]:
        ys, ds = [o], [s["do"].float()]
        if s["dS"] is not None:
            ys, ds = ys + [S], ds + [s["dS"]]
        for n, d in zip(names, torch.autograd.grad(ys, [x[n] for n in names], ds)):
            out["d" + n] = d.to(s[n].dtype)
    return out


def _plain_step(s):
    r = s["Hv"] // s["Hk"]
    q = s["q"].float().repeat_interleave(r, 1)
    k = s["k"].float().repeat_interleave(r, 1)
    slots = s["slots"].long()
    S = s["pool_state"][slots] * torch.exp(s["gk"])[..., None, None]
    u = s["beta"].float()[..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    o = s["scale"] * (S * q[..., None]).sum(-2)
    s["pool_state"][slots] = S
    return {"o": o.bfloat16(), "state": s["pool_state"]}


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        return _own(s)
    return {"block": _plain_block, "delta": _plain_delta, "step": _plain_step}[s["op"]](s)


def _own(s):
    import gated_norm_b200 as gn

    if s["op"] == "step":
        o = gn.gnorm_delta_step(s["q"], s["k"], s["v"], s["gk"], s["beta"], s["pool_state"],
                                slots=s["slots"], scale=s["scale"])
        return {"o": o, "state": s["pool_state"]}
    if s["op"] == "block":
        h, z, rstd1, rstd2 = gn.gnorm_block_fwd(s["a"], s["r"], s["w1"], s["w2"], EPS,
                                                g=s["g"], alpha=s["alpha"])
        out = {"h": h, "z": z}
        if s["train"]:
            da, dr, dg, dw1, dw2, dalpha = gn.gnorm_block_bwd(
                s["dh"], s["dz"], s["a"], s["r"], s["w1"], s["w2"], rstd1, rstd2, g=s["g"],
                alpha=s["alpha"], dw_fp32=True)
            out |= {"da": da, "dr": dr, "dw1": dw1, "dw2": dw2, "dalpha": dalpha}
            if dg is not None:
                out["dg"] = dg
        return out
    train, state = s["train"], s["S0"] is not None
    o, S = gn.gnorm_delta_fwd(s["q"], s["k"], s["v"], s["gk"], s["beta"], scale=s["scale"],
                              cu_seqlens=s["cu"], initial_state=s["S0"],
                              output_final_state=state or not train)
    out = {"o": o}
    if S is not None:
        out["state"] = S
    if train:
        dq, dk, dv, dg, dbeta, dS0 = gn.gnorm_delta_bwd(
            s["do"], s["q"], s["k"], s["v"], s["gk"], s["beta"], scale=s["scale"],
            cu_seqlens=s["cu"], initial_state=s["S0"], dfinal_state=s["dS"])
        out |= {"dq": dq, "dk": dk, "dv": dv, "dgk": dg, "dbeta": dbeta}
        if state:
            out["dS0"] = dS0
    return out


# ------------------------------------------------------- the definition, in 64 bits

def _exact_block(s):
    d = {n: None if s.get(n) is None else s[n].double()
         for n in ("a", "r", "g", "alpha", "w1", "w2", "dh", "dz")}
    N = s["N"]
    r1 = (d["a"].square().sum(-1, keepdim=True) / N + EPS) ** -0.5
    ah = d["a"] * r1
    b = ah * d["w1"]
    sg = None if d["g"] is None else 1.0 / (1.0 + torch.exp(-d["g"]))
    silu = 1.0 if sg is None else d["g"] * sg
    h = d["r"] + d["alpha"] * silu * b
    r2 = (h.square().sum(-1, keepdim=True) / N + EPS) ** -0.5
    hh = h * r2
    out = {"h": h, "z": hh * d["w2"]}
    if s["train"]:
        u2 = d["dz"] * d["w2"]
        dh = d["dh"] + r2 * (u2 - hh * (u2 * hh).sum(-1, keepdim=True) / N)
        out["dw2"] = (d["dz"] * hh).sum(0)
        out["dr"] = dh
        out["dalpha"] = (dh * silu * b).sum().reshape(1)
        db = d["alpha"] * dh * silu
        out["dw1"] = (db * ah).sum(0)
        u1 = db * d["w1"]
        out["da"] = r1 * (u1 - ah * (u1 * ah).sum(-1, keepdim=True) / N)
        if sg is not None:
            out["dg"] = d["alpha"] * dh * b * sg * (1.0 + d["g"] * (1.0 - sg))
    return out


def _exact_delta(s):
    """The recurrence token by token, and its adjoint; states are kept at every 64th token and
    computed again in between."""
    T, Hk, K = s["q"].shape
    Hv, V = s["v"].shape[1:]
    B, L, r, dev = s["B"], s["max_len"], s["Hv"] // s["Hk"], s["q"].device
    cu = s["cu"].long()
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    p = t - cu[b]

    def lay(x, heads):  # time first: [L, B, Hv, D]; nothing happens behind a sequence's end
        y = torch.zeros(L, B, x.shape[1], x.shape[2], dtype=torch.float64, device=dev)
        y[p, b] = x.double()
        return y.repeat_interleave(heads, 2)

    q, k, v = lay(s["q"], r), lay(s["k"], r), lay(s["v"], 1)
    w = torch.exp(lay(s["gk"][..., None], 1))[..., None]
    beta = lay(s["beta"][..., None], 1)
    S = torch.zeros(B, Hv, K, V, dtype=torch.float64, device=dev) if s["S0"] is None \
        else s["S0"].double()
    o = torch.zeros(L, B, Hv, V, dtype=torch.float64, device=dev)
    kept = []

    def step(S, i):
        S = S * w[i]
        u = beta[i] * (v[i] - (k[i][..., None, :] @ S)[..., 0, :])
        return S + k[i][..., None] * u[..., None, :]

    for i in range(L):
        if i % CHUNK == 0:
            kept.append(S)
        S = step(S, i)
        o[i] = s["scale"] * (q[i][..., None, :] @ S)[..., 0, :]
    out = {"o": o[p, b]}
    if not s["train"] or s["S0"] is not None:
        out["state"] = S
    if not s["train"]:
        return out
    do = s["scale"] * lay(s["do"], 1)
    dS = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dw, dbeta = torch.zeros_like(beta), torch.zeros_like(beta)
    for c in reversed(range(len(kept))):
        hi = min(L, (c + 1) * CHUNK)
        before = [kept[c]]
        for i in range(c * CHUNK, hi):
            before.append(step(before[-1], i))
        for i in reversed(range(c * CHUNK, hi)):
            St, Sd = before[i - c * CHUNK + 1], before[i - c * CHUNK] * w[i]
            dq[i] = (St @ do[i][..., None])[..., 0]
            dS = dS + q[i][..., None] * do[i][..., None, :]
            e = v[i] - (k[i][..., None, :] @ Sd)[..., 0, :]
            du = (k[i][..., None, :] @ dS)[..., 0, :]
            dbeta[i] = (du * e).sum(-1, keepdim=True)
            de = beta[i] * du
            dv[i] = de
            dk[i] = (dS @ (beta[i] * e)[..., None])[..., 0] - (Sd @ de[..., None])[..., 0]
            dS = dS - k[i][..., None] * de[..., None, :]
            dw[i] = (dS * Sd).sum((-1, -2))[..., None]  # d/dg of exp(g) S is exp(g) S
            dS = dS * w[i]

    def heads(x):
        return x[p, b].reshape(T, Hk, r, -1).sum(2)

    out |= {"dq": heads(dq), "dk": heads(dk), "dv": dv[p, b], "dgk": dw[p, b][..., 0],
            "dbeta": dbeta[p, b][..., 0]}
    if s["S0"] is not None:
        out["dS0"] = dS
    return out


def _exact_step(s):
    r = s["Hv"] // s["Hk"]
    pool = s["pool_state"].double()
    o = torch.empty(s["v"].shape, dtype=torch.float64, device=pool.device)
    for h in range(s["Hv"]):
        S = pool[s["slots"].long(), h] * s["gk"][:, h].double().exp()[:, None, None]
        k, q = s["k"][:, h // r].double(), s["q"][:, h // r].double()
        u = s["beta"][:, h, None].double() * (s["v"][:, h].double() -
                                              torch.einsum("bk,bkv->bv", k, S))
        S = S + torch.einsum("bk,bv->bkv", k, u)
        o[:, h] = s["scale"] * torch.einsum("bk,bkv->bv", q, S)
        pool[s["slots"].long(), h] = S
    return {"o": o, "state": pool}


def exact(case, seed):
    s = prepare(case, seed)
    return {"block": _exact_block, "delta": _exact_delta, "step": _exact_step}[s["op"]](s)
