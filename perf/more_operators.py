"""Workloads of the gated delta rule and of group norm, each for prompts or
maps, for training and for single tokens, in plain torch operations and through
this package's kernels.

The gated delta rule keeps a K x V matrix S for each sequence and head:

    d = softplus(dt + dt_bias),  a = exp(d * A),  b = sigmoid(beta)
    q, k = q / sqrt(sum q^2 + 1e-6), k / sqrt(sum k^2 + 1e-6)
    S = a * S;  S = S + b * k (v - k S);  y = scale * q S

Group norm is over [N, ..., C] with the channels last: a mean and a variance
for each n and group of C/G neighbouring channels, then
y = act(h * gamma + beta) * silu(z), the gate z where it is given.

A batch of sequences is dense ([S, L, ...]) or packed ([T, ...] with
``offsets``); sequences of no token and of one token are among the packed ones.
Parameters and states are fp32, activations of the case's type.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
QK_EPS = 1e-6
CHUNK = 64


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # Four prompts of 4096 tokens through a layer of 16 heads.
        dict(name="delta_prompt_bf16", op="delta", mode="prompt", dtype="bf16", seqs=4, tokens=16384, HK=16, HV=16,
             K=128, V=128, packed=False, state=False),
        # One long sequence alone, in fp32: few rows, a long axis.
        dict(name="delta_long_f32", op="delta", mode="prompt", dtype="f32", seqs=1, tokens=16384, HK=8, HV=8, K=64,
             V=64, packed=False, state=False),
        # The next chunks of 9 prompts of many lengths, continued from their
        # states; two value heads for each key head, odd sizes.
        dict(name="delta_chunk_f16", op="delta", mode="prompt", dtype="f16", seqs=9, tokens=3137, HK=4, HV=8, K=96,
             V=81, packed=True, state=True),
        # A training step, forward and backward, shared key heads.
        dict(name="delta_train_bf16", op="delta", mode="train", dtype="bf16", seqs=2, tokens=4096, HK=8, HV=16, K=128,
             V=128, packed=False, state=False),
        # Training on packed sequences of many lengths, small odd heads.
        dict(name="delta_train_f16", op="delta", mode="train", dtype="f16", seqs=13, tokens=2001, HK=6, HV=6, K=64,
             V=50, packed=True, state=False),
        # One token for each of 64 running sequences, their states in a cache.
        dict(name="delta_step_bf16", op="delta", mode="step", dtype="bf16", seqs=64, HK=16, HV=16, K=128, V=128),
        # One token for each of 2 sequences: latency is all that counts.
        dict(name="delta_step_f16", op="delta", mode="step", dtype="f16", seqs=2, HK=4, HV=8, K=128, V=128),
        # The 56x56 maps of 32 images, the norm and SiLU before a convolution.
        dict(name="gnorm_maps_f16", op="gnorm", mode="infer", dtype="f16", N=32, L=3136, C=256, G=32, act="silu", gate=False),
        # Training on 56x56 maps, forward and backward.
        dict(name="gnorm_train_bf16", op="gnorm", mode="train", dtype="bf16", N=16, L=3136, C=128, G=32, act="silu", gate=False),
        # Training in fp32 on 19x19 maps, at widths that are no multiple of anything.
        dict(name="gnorm_train_f32", op="gnorm", mode="train", dtype="f32", N=9, L=361, C=363, G=3, act="silu", gate=False),
        # The norm of each token's heads with its gate, behind the delta rule, in training.
        dict(name="gnorm_heads_bf16", op="gnorm", mode="train", dtype="bf16", N=16384, L=1, C=2048, G=16, act="none", gate=True),
        # The same for one token of each of 64 sequences.
        dict(name="gnorm_step_f16", op="gnorm", mode="infer", dtype="f16", N=64, L=1, C=2048, G=16, act="none", gate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, mode = rng.choice([("delta", "prompt"), ("delta", "prompt"), ("delta", "train"), ("delta", "train"), ("delta", "step"),
                           ("gnorm", "infer"), ("gnorm", "train"), ("gnorm", "train")])
    c = dict(op=op, mode=mode, dtype=rng.choice(["f16", "bf16", "f32"]))
    if op == "gnorm":
        heads = rng.random() < 0.4
        G = rng.choice([1, 2, 3, 4, 8, 16, 32])
        C = G * _log(rng, 16, 256) if heads else G * max(1, _log(rng, 32, 1024) // G)
        L = 1 if heads else _log(rng, 4, 4096)
        top = (1 << 25) if mode == "infer" else (1 << 24)
        N = max(1, min(_log(rng, 1, 16384 if heads else 64), top // (L * C)))
        return dict(c, N=N, L=L, C=C, G=G, act=rng.choice(["silu", "silu", "none"]), gate=heads and rng.random() < 0.7)
    HK = rng.choice([1, 2, 3, 4, 8, 16])
    HV = HK * rng.choice([1, 1, 2, 4]) if HK <= 8 else HK
    K, V = _log(rng, 16, 256), _log(rng, 16, 256)
    if rng.random() < 0.6:
        K, V = rng.choice([64, 128]), rng.choice([64, 128, 256])
    c.update(HK=HK, HV=HV, K=K, V=V)
    if mode == "step":
        return dict(c, seqs=min(_log(rng, 1, 256), max(1, (1 << 24) // (HV * K * V))))
    top = (15 << 28) if mode == "prompt" else (15 << 26)
    seqs = _log(rng, 1, 24)
    tokens = min(_log(rng, max(seqs, 16), 16384), max(seqs, top // (HV * K * V)))
    packed = rng.random() < 0.5
    if not packed:
        tokens -= tokens % seqs
    return dict(c, seqs=seqs, tokens=tokens, packed=packed, state=mode == "prompt" and rng.random() < 0.5)


# --------------------------------------------------------------- the inputs

def _lengths(case, gen):
    """Lengths of packed sequences: log-uniform shares, an empty one and one
    of a single token among them where there are at least four."""
    S, T = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [T // S] * S
    share = torch.exp(3.0 * torch.rand(S, generator=gen, device="cpu"))
    n = [int(v) for v in torch.floor(share / share.sum() * T)]
    if S >= 4 and T >= 2 * S:
        n[1], n[S // 2] = 0, 1
    n[S - 1] += T - sum(n)
    return n


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator(device="cpu").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale + shift).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    f32 = torch.float32
    s = dict(case=case)
    if case["op"] == "gnorm":
        N, L, C = case["N"], case["L"], case["C"]
        shape = (N, C) if L == 1 else (N, L, C)
        s["x"] = randn(*shape, scale=1.5, shift=0.3)
        s["z"] = randn(*shape) if case["gate"] else None
        s["gamma"], s["beta"] = randn(C, scale=0.2, shift=1.0, dtype=f32), randn(C, scale=0.2, dtype=f32)
        if case["mode"] == "train":
            s["dy"] = randn(*shape)
        return s

    S, HK, HV, K, V = (case[k] for k in ("seqs", "HK", "HV", "K", "V"))
    if case["mode"] == "step":
        lead = (S,)
        # The sequences' places in a cache that has room for more of them.
        s["slots"] = torch.randperm(S + 7, generator=cpu)[:S].to(torch.int32).to(dev)
        s["state"] = randn(S + 7, HV, K, V, scale=0.3, dtype=f32)
    else:
        T, n = case["tokens"], _lengths(case, cpu)
        lead = (T,) if case["packed"] else (S, T // S)
        s["lengths"] = n
        s["bounds"] = torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(dev)
        s["offsets"] = s["bounds"].to(torch.int32) if case["packed"] else None
        s["state"] = randn(S, HV, K, V, scale=0.3, dtype=f32) if case["state"] else None
        if case["mode"] == "train":
            s["dy"] = randn(*lead, HV, V)
    # q, k and v are slices of one projection's output.
    qkv = randn(*lead, 2 * HK * K + HV * V)
    s["q"] = qkv[..., :HK * K].unflatten(-1, (HK, K))
    s["k"] = qkv[..., HK * K:2 * HK * K].unflatten(-1, (HK, K))
    s["v"] = qkv[..., 2 * HK * K:].unflatten(-1, (HV, V))
    # Step sizes around 0.001 to 0.1, decay rates from 1 to 16.
    step = torch.exp(rand(HV) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = randn(*lead, HV, scale=0.5)
    s["A"] = -(1 + 15 * rand(HV))
    s["beta"] = randn(*lead, HV)
    return s


def work(case):
    """Bytes: each input read once, each output written once. Operations: the
    formulas' multiplications, additions and exponentials, one each. The delta
    rule's are those of the recurrence (three products of the state with a
    vector for each token, and the decay), twice and a half as many more with
    the backward pass."""
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "gnorm":
        n, C, z = case["N"] * case["L"] * case["C"], case["C"], case["gate"]
        b, f = n * e * (3 if z else 2) + 8 * C, n * (16 if z else 12)
        if case["mode"] == "train":
            b, f = b + n * e * (3 if z else 2) + 8 * C, f + n * (34 if z else 24)
        return {"bytes": b, "flops": f}
    S, HK, HV, K, V = (case[k] for k in ("seqs", "HK", "HV", "K", "V"))
    rows = S if case["mode"] == "step" else case["tokens"]
    token = (2 * HK * K + 2 * HV * V + 2 * HV) * e
    held = S * HV * K * V * 4
    b, f = rows * token + 8 * HV, rows * HV * (7 * K * V + 8 * K + 4 * V)
    if case["mode"] == "train":
        b, f = b + rows * token + 8 * HV, f + rows * HV * (17 * K * V + 20 * K + 10 * V)
    elif case["mode"] == "step":
        b += 2 * held
    else:
        b += held * (2 if case["state"] else 1)
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------- the plain form

def _silu_slope(v):
    sg = torch.sigmoid(v)
    return sg * (1 + v * (1 - sg))


def _plain_gnorm(s):
    case, td = s["case"], s["x"].dtype
    N, L, C, G = (case[k] for k in ("N", "L", "C", "G"))
    shape, silu = s["x"].shape, case["act"] == "silu"

    def groups(v):
        return v.reshape(N, L, G, C // G)

    def mean(v):
        return v.mean((1, 3), keepdim=True)

    x = groups(s["x"].float())
    d = x - mean(x)
    r = torch.rsqrt(mean(d * d) + EPS)
    h = d * r
    gamma = s["gamma"].reshape(G, C // G)
    v = h * gamma + s["beta"].reshape(G, C // G)
    a = v * torch.sigmoid(v) if silu else v
    z = None if s["z"] is None else groups(s["z"].float())
    y = a if z is None else a * z * torch.sigmoid(z)
    y = y.reshape(shape).to(td)
    if case["mode"] == "infer":
        return [y]
    da, dz = groups(s["dy"].float()), None
    if z is not None:
        dz = (da * a * _silu_slope(z)).reshape(shape).to(td)
        da = da * z * torch.sigmoid(z)
    dv = da * _silu_slope(v) if silu else da
    g = dv * gamma
    dx = r * (g - mean(g) - h * mean(g * h))
    return [y, dx.reshape(shape).to(td), (dv * h).sum((0, 1)).reshape(C), dv.sum((0, 1)).reshape(C), dz]


def _gates(s):
    """The step size's slope and d, the decay's logarithm and b, fp32."""
    raw = s["dt"].float() + s["dt_bias"]
    d = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw)))
    return raw, d, d * s["A"], torch.sigmoid(s["beta"].float())


def _unit(x):
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) + QK_EPS)
    return x * r, r


def _plain_delta_step(s):
    case, at = s["case"], s["slots"].long()
    rep, scale = case["HV"] // case["HK"], case["K"] ** -0.5
    _, _, g, b = _gates(s)
    q, k = (_unit(s[n].float())[0].repeat_interleave(rep, 1) for n in ("q", "k"))
    S = s["state"][at] * torch.exp(g)[..., None, None]
    u = b[..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    y = scale * (q[..., None] * S).sum(-2)
    s["state"][at] = S
    return [y.to(s["v"].dtype), s["state"]]


def _mm(a, b):
    return torch.matmul(a.contiguous(), b.contiguous())


def _plain_delta(s):
    """In chunks of 64 tokens. With G the decays' logarithms added up from the
    chunk's first token, D[i, j] = exp(G[i] - G[j]) for j <= i and S0 the state
    before the chunk, the corrections E[i] = v[i] - k[i] (decayed S) solve
        (I + N) E = v - exp(G) k S0,   N[i, j] = D[i, j] (k[i] k[j]) b[j], j < i
    and y = scale (exp(G) q S0 + (D * q k^T) b E)."""
    case, td, dev = s["case"], s["v"].dtype, s["v"].device
    S, HK, HV, K, V = (case[n] for n in ("seqs", "HK", "HV", "K", "V"))
    rep, scale, T = HV // HK, case["K"] ** -0.5, case["tokens"]
    lengths = s["lengths"]
    C = CHUNK
    n = max(1, -(-max(lengths) // C))
    # Rows of a batch padded to whole chunks; row T stands for none.
    at = s["bounds"][:-1, None] + torch.arange(n * C, device=dev)
    at = torch.where(at < s["bounds"][1:, None], at, T)

    def chunks(v, fill=0.0):  # [rows, H, W] -> [S, H, n, C, W]
        v = torch.cat([v, torch.full_like(v[:1], fill)])[at]
        return v.reshape(S, n, C, v.shape[-2], v.shape[-1]).permute(0, 3, 1, 2, 4)

    def rows(v):  # and back
        v = v.permute(0, 2, 3, 1, 4).reshape(S * n * C, v.shape[1], v.shape[-1])
        out = torch.empty(T + 1, v.shape[1], v.shape[2], dtype=v.dtype, device=dev)
        out[at.reshape(-1)] = v
        return out[:T]

    raw, d, g, b = (v.reshape(T, HV, 1) for v in _gates(s))
    q0, k0 = s["q"].reshape(T, HK, K).float(), s["k"].reshape(T, HK, K).float()
    (qn, rq), (kn, rk) = _unit(q0), _unit(k0)
    q, k = (chunks(v).repeat_interleave(rep, 1) for v in (qn, kn))
    v, b = chunks(s["v"].reshape(T, HV, V).float()), chunks(b)
    G = chunks(g).double().cumsum(-2)
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    D = torch.exp(torch.where(low, G - G.transpose(-1, -2), -math.inf)).float()
    eG, tail = torch.exp(G).float(), torch.exp(G[..., -1:, :] - G).float()
    kk, P = _mm(k, k.transpose(-1, -2)) * D, _mm(q, k.transpose(-1, -2)) * D * scale
    Lh = kk.tril(-1)
    Nm = Lh * b.transpose(-1, -2)
    X = torch.eye(C, device=dev).expand(Nm.shape).clone()  # (I + N)^-1 by rows
    for i in range(1, C):
        X[..., i, :i] = -_mm(Nm[..., i:i + 1, :i], X[..., :i, :i])[..., 0, :]
    state = torch.zeros(S, HV, K, V, device=dev) if s["state"] is None else s["state"]
    train = case["mode"] == "train"
    starts, Es, ys = [], [], []
    for c in range(n):
        starts.append(state)
        E = _mm(X[:, :, c], v[:, :, c] - eG[:, :, c] * _mm(k[:, :, c], state))
        U = b[:, :, c] * E
        ys.append(scale * eG[:, :, c] * _mm(q[:, :, c], state) + _mm(P[:, :, c], U))
        state = eG[:, :, c, -1:] * state + _mm((tail[:, :, c] * k[:, :, c]).transpose(-1, -2), U)
        Es.append(E)
    lead = s["v"].shape[:-2]
    y = rows(torch.stack(ys, 2)).reshape(lead + (HV, V)).to(td)
    if not train:
        return [y, state]
    # Backward, chunk by chunk from the last: R is the gradient of v.
    dy = chunks(s["dy"].reshape(T, HV, V).float())
    dS = torch.zeros_like(state)
    dqs, dks, dvs, dbs, dgs = ([None] * n for _ in range(5))
    for c in reversed(range(n)):
        qc, kc, bc, e, t, S0, E, w = q[:, :, c], k[:, :, c], b[:, :, c], eG[:, :, c], tail[:, :, c], starts[c], Es[c], dy[:, :, c]
        kS = _mm(kc, dS) * t
        dU = _mm(P[:, :, c].transpose(-1, -2), w) + kS
        R = _mm(X[:, :, c].transpose(-1, -2), bc * dU)
        F, H = _mm(w, E.transpose(-1, -2)), -_mm(R, E.transpose(-1, -2))
        qS, RS, ES = (_mm(m, s_.transpose(-1, -2)) for m, s_ in ((w, S0), (R, S0), (E, dS)))
        bt = bc.transpose(-1, -2)
        dP, M = F * bt * D[:, :, c] * scale, H * bt * D[:, :, c].tril(-1)
        dqs[c] = scale * e * qS + _mm(dP, kc)
        dks[c] = _mm(dP.transpose(-1, -2), qc) + t * bc * ES - e * RS + _mm(M + M.transpose(-1, -2), kc)
        dvs[c] = R
        Z = (kS * E).sum(-1, keepdim=True)
        dbs[c] = Z + (P[:, :, c] * F + Lh[:, :, c] * H).sum(-2).unsqueeze(-1)
        pair = bt * (P[:, :, c] * F + Lh[:, :, c] * H)
        dG = pair.sum(-1, keepdim=True) - pair.sum(-2).unsqueeze(-1) - bc * Z + e * ((scale * qc * qS) - kc * RS).sum(-1, keepdim=True)
        dG[..., -1, :] += (e[..., -1, :] * (dS * S0).sum((-1, -2)).unsqueeze(-1) + (bc * Z).sum(-2))
        dgs[c] = dG.flip(-2).cumsum(-2).flip(-2)
        dS = e[..., -1:, :] * dS + _mm((scale * e * qc).transpose(-1, -2), w) - _mm((e * kc).transpose(-1, -2), R)

    def raw_of(parts, x, r):  # over the value heads of a key head, then through the length
        dx = rows(torch.stack(parts, 2)).reshape(T, HK, rep, K).sum(2)
        return (r * (dx - x * (x * dx).sum(-1, keepdim=True))).reshape(lead + (HK, K)).to(td)

    dg = rows(torch.stack(dgs, 2))[..., 0]
    draw_ = dg * s["A"] * torch.sigmoid(raw[..., 0])
    sb = torch.sigmoid(s["beta"].reshape(T, HV).float())
    db = rows(torch.stack(dbs, 2))[..., 0] * sb * (1 - sb)
    dv = rows(torch.stack(dvs, 2)).reshape(lead + (HV, V)).to(td)
    return [y, raw_of(dqs, qn, rq), raw_of(dks, kn, rk), dv, draw_.reshape(lead + (HV,)).to(td),
            (dg * d[..., 0]).sum(0), db.reshape(lead + (HV,)).to(td), draw_.sum(0)]


# ------------------------------------------------- through the own kernels

def _own_gnorm(s):
    import conv2d_batchnorm_silu_amd as tg
    case = s["case"]
    more = dict(eps=EPS, act=case["act"], z=s["z"])
    if case["mode"] == "infer":
        return [tg.group_norm(s["x"], case["G"], s["gamma"], s["beta"], **more)]
    y, mean, rstd = tg.group_norm_train(s["x"], case["G"], s["gamma"], s["beta"], **more)
    d = tg.group_norm_backward(s["dy"], s["x"], case["G"], s["gamma"], mean, rstd, beta=s["beta"], act=case["act"], z=s["z"])
    return [y, d.dx, d.dgamma, d.dbeta, d.dz]


def _own_delta(s):
    import conv2d_batchnorm_silu_amd as tg
    mode = s["case"]["mode"]
    args = (s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"])
    if mode == "step":
        return [tg.gated_delta_rule_step(*args, s["state"], dt_bias=s["dt_bias"], slots=s["slots"]), s["state"]]
    more = dict(dt_bias=s["dt_bias"], offsets=s["offsets"])
    if mode == "prompt":
        return list(tg.gated_delta_rule(*args, initial_state=s["state"], return_state=True, **more))
    y, saved = tg.gated_delta_rule_train(*args, **more)
    d = tg.gated_delta_rule_backward(s["dy"], *args, saved, **more)
    return [y, d.dq, d.dk, d.dv, d.ddt, d.dA, d.dbeta, d.ddt_bias]


def run(state):
    case = state["case"]
    if own:
        return (_own_gnorm if case["op"] == "gnorm" else _own_delta)(state)
    if case["op"] == "gnorm":
        return _plain_gnorm(state)
    return _plain_delta_step(state) if case["mode"] == "step" else _plain_delta(state)


# ------------------------------------------------------ by definition, fp64

def _exact_gnorm(s):
    case = s["case"]
    train, G = case["mode"] == "train", case["G"]
    x, gamma, beta = (s[n].double().requires_grad_(train) for n in ("x", "gamma", "beta"))
    z = None if s["z"] is None else s["z"].double().requires_grad_(train)
    parts = []
    for xs, ga, be in zip(x.chunk(G, -1), gamma.chunk(G), beta.chunk(G)):
        every = tuple(range(1, x.dim()))
        var, mean = torch.var_mean(xs, every, unbiased=False, keepdim=True)
        parts.append((xs - mean) / torch.sqrt(var + EPS) * ga + be)
    y = torch.cat(parts, -1)
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if z is not None:
        y = y * z / (1 + torch.exp(-z))
    if not train:
        return [y]
    leaves = [x, gamma, beta] + ([] if z is None else [z])
    d = list(torch.autograd.grad(y, leaves, s["dy"].double()))
    return [y.detach()] + d + ([None] if z is None else [])


def _exact_delta(s):
    case = s["case"]
    HK, HV, K, V = (case[n] for n in ("HK", "HV", "K", "V"))
    train, rep = case["mode"] == "train", HV // HK
    q, k, v, dt, A, beta, bias = (s[n].double().requires_grad_(train) for n in ("q", "k", "v", "dt", "A", "beta", "dt_bias"))
    raw = dt + bias
    a = torch.exp(A * (torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))))
    b = 1 / (1 + torch.exp(-beta))
    qn, kn = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + QK_EPS) for x in (q, k))
    qn, kn = (x.unsqueeze(-2).expand(x.shape[:-1] + (rep, K)).flatten(-3, -2) for x in (qn, kn))

    def token(S, qt, kt, vt, at, bt):  # [n, HV, ...]
        S = at[..., None, None] * S
        u = bt[..., None] * (vt - (kt.unsqueeze(-2) @ S).squeeze(-2))
        S = S + kt.unsqueeze(-1) * u.unsqueeze(-2)
        return S, (qt.unsqueeze(-2) @ S).squeeze(-2)

    if case["mode"] == "step":
        state, at = s["state"].double().clone(), s["slots"].long()
        state[at], y = token(state[at], qn, kn, v, a, b)
        return [y * K ** -0.5, state]
    zero = torch.zeros(case["seqs"], HV, K, V, dtype=torch.float64, device=v.device)
    S = zero if s["state"] is None else s["state"].double()
    if case["packed"]:
        ys, last, t = [], [], 0
        for i, n in enumerate(s["lengths"]):
            h = S[i:i + 1]
            for t in range(t, t + n):
                h, y = token(h, qn[t:t + 1], kn[t:t + 1], v[t:t + 1], a[t:t + 1], b[t:t + 1])
                ys.append(y)
            t = len(ys)
            last.append(h.detach())
        y, S = torch.cat(ys), torch.cat(last)
    else:
        ys = []
        for t in range(v.shape[1]):
            S, y = token(S, qn[:, t], kn[:, t], v[:, t], a[:, t], b[:, t])
            ys.append(y)
        y, S = torch.stack(ys, 1), S.detach()
    y = y * K ** -0.5
    if not train:
        return [y, S]
    dq, dk, dv, ddt, dA, dbeta, dbias = torch.autograd.grad(y, [q, k, v, dt, A, beta, bias], s["dy"].double())
    return [y.detach(), dq, dk, dv, ddt, dA, dbeta, dbias]


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_gnorm if case["op"] == "gnorm" else _exact_delta)(s)
