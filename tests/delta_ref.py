"""References of the gated delta rule and of group norm in 64 bits, from the
formulas of include/tg_sequence.h, and what the kernels may be off.

The delta rule. With unit keys and 0 <= b <= 1 a token's map of the state has no
norm above one, so errors do not grow from token to token; what a chunk of C tokens
adds is amplified by the inverse X of its triangular matrix, whose norm KAPPA is
taken from the inputs. On the way from one chunk's state to the next lie fewer than
STEPS = 32 roundings (the parts of S, v - k S, the factors of rows, the parts of the
right side, X by substitution in 16 steps and two block products, the corrections'
factors and parts, the sums in the matrix instructions), each of u relative: 2^-18
where operands are two bf16 parts (prompts of 16-bit tensors), 2^-24 else. So a state after n chunks is off by n * STEPS * KAPPA * u of its norm and of what was
added to it, and the gradients, which go through both walks, by twice that with
KAPPA^2. y of 16-bit tensors is made of products of two parts, three operands of 2^-17
(a part's rounding and the dropped product of two second parts); the pairs' part of
dq and dk of as many parts as an input has, 2^-9 for bf16. Every output adds half a
step of its type. A single element is held to 8 times that of the
root mean square (or of itself where it is larger): four standard deviations of a
sum of many roundings, twice. Sums over all tokens (dA, ddt_bias) cancel: they are
held against the sum of the magnitudes."""
from __future__ import annotations

import torch

E = 2.0 ** -24
F64 = torch.float64
STEPS = 32


def gates(dt, A, beta, dt_bias, softplus, sigmoid):
    raw = dt if dt_bias is None else dt + dt_bias
    d = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    g = torch.where(d == 0, torch.zeros_like(d), A * d)
    return d, g, torch.sigmoid(beta) if sigmoid else beta


def unit(x, normalize):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) if normalize else x


def walk(q, k, v, g, b, scale, S):
    """One sequence, token by token: q, k [L, HV, K], v [L, HV, V], g, b [L, HV],
    S [HV, K, V] -> (y [L, HV, V], S)."""
    ys = []
    for t in range(v.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S
        u = b[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t][:, :, None] * u[:, None, :]
        ys.append(scale * torch.einsum("hk,hkv->hv", q[t], S))
    return torch.stack(ys) if ys else torch.zeros_like(v), S


def kappa(k, g, b, C):
    """The largest norm of a chunk's X, from its N."""
    worst = 1.0
    for lo in range(0, k.shape[0], C):
        # A decay of e^-200 is none in fp32; an infinite one has no differences.
        kc, G, bc = k[lo:lo + C], g[lo:lo + C].clamp(min=-200).cumsum(0), b[lo:lo + C]
        for h in range(k.shape[1]):
            N = (torch.exp(G[:, None, h] - G[None, :, h]) * (kc[:, h] @ kc[:, h].t()) * bc[None, :, h]).tril(-1)
            X = torch.linalg.inv(torch.eye(N.shape[0], dtype=F64) + N)
            worst = max(worst, float(torch.linalg.matrix_norm(X, 2)))
    return worst


def spread(x, HV):
    return x.repeat_interleave(HV // x.shape[-2], -2)


def delta(bounds, q, k, v, dt, A, beta, dt_bias=None, softplus=True, sigmoid=True, normalize=True, scale=None,
          initial=None):
    """y, the final states [S, HV, K, V], the decays' logarithms and the unit q and k of
    packed rows; also KAPPA and the most chunks of a sequence."""
    HV, K = v.shape[-2], k.shape[-1]
    scale = K ** -0.5 if scale is None else scale
    d, g, b = gates(dt, A, beta, dt_bias, softplus, sigmoid)
    units = unit(q, normalize), unit(k, normalize)
    qn, kn = spread(units[0], HV), spread(units[1], HV)
    ys, states, worst, most = [], [], 1.0, 1
    for i, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        S = torch.zeros(HV, K, v.shape[-1], dtype=F64) if initial is None else initial[i]
        y, S = walk(qn[lo:hi], kn[lo:hi], v[lo:hi], g[lo:hi], b[lo:hi], scale, S)
        ys.append(y)
        states.append(S)
        with torch.no_grad():
            worst = max(worst, kappa(kn[lo:hi].detach(), g[lo:hi].detach(), b[lo:hi].detach(), 64))
        most = max(most, -(-(hi - lo) // 32))
    return torch.cat(ys), torch.stack(states), (g, *units), worst, most


def near(name, got, want, rel, dtype, size=None):
    """2-norm and single elements, as above; ``size``: what an element is a sum of."""
    g, w = got.detach().double().cpu(), want.detach()
    assert g.shape == w.shape, (name, g.shape, w.shape)
    if w.numel() == 0:
        return
    half = torch.finfo(dtype).eps / 2
    mag = w.abs() if size is None else torch.maximum(w.abs(), size)
    d = (g - w).abs()
    norm, whole = float(d.norm()), float(mag.norm())
    assert norm <= (rel + half) * whole + 1e-30, "%s: %.3g of %.3g, allowed %.3g" % (name, norm, whole, rel + half)
    rms = mag.norm() / mag.numel() ** 0.5
    worst = float((d / torch.maximum(mag, rms)).max()) if whole else float(d.max())
    assert worst <= 8 * rel + 2 * half, "%s: an element off by %.3g, allowed %.3g" % (name, worst, 8 * rel + 2 * half)


def allowed(dtype, kap, chunks, gradient=False, only=None, prompt=False):
    """Relative error of an output, without its own rounding; ``only``: "y" or "qk",
    what is made of fewer parts; ``prompt``: without training."""
    u = 2.0 ** -18 if prompt and dtype is not torch.float32 else E
    rel = 2 * chunks * STEPS * kap * kap * u if gradient else chunks * STEPS * kap * u
    if only and dtype is not torch.float32:
        rel += 3 * (2.0 ** -9 if only == "qk" and dtype is torch.bfloat16 else 2.0 ** -17)
    return rel


def unit_size(x, dunit):
    """What an element of the gradient of x is a difference of, where x enters through
    n = r x: dx = D - n (n.D) with D = r dn, and |n| <= 1, so its two terms are |D| and
    at most |n| |D|, of which all roundings before the subtraction are a share."""
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)
    d = (r * dunit).detach()
    return (d.abs() + (r * x).detach().abs() * d.norm(dim=-1, keepdim=True))


# ---- group norm

def group_norm(x, G, gamma, beta, eps, act, z):
    """y, mean, rstd of x [N, L, C] (64-bit, differentiable)."""
    N, L, C = x.shape
    v = x.reshape(N, L, G, C // G)
    mean = v.mean((1, 3), keepdim=True)
    d = v - mean
    rstd = 1 / torch.sqrt((d * d).mean((1, 3), keepdim=True) + eps)
    y = (d * rstd).reshape(N, L, C) * gamma + (0 if beta is None else beta)
    if act == "silu":
        y = y * torch.sigmoid(y)
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y, mean.reshape(N, G), rstd.reshape(N, G)


def group_bounds(x, G, eps):
    """What mean, rstd and h may be off: the mean by 64 roundings of its own size and
    of the mean distance (sums of 32, joins of sets), the sum of squares by 32 times
    four roundings (its subtraction), 64 of joins, and what the means' errors
    add where they are large against the spread."""
    N, L, C = x.shape
    v = x.reshape(N, L, G, C // G)
    mean = v.mean((1, 3), keepdim=True)
    d = v - mean
    var = (d * d).mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    emean = 64 * E * (mean.abs() + 2 * d.abs().mean((1, 3), keepdim=True))
    ers = E * (100 + 8 * mean.abs() * rstd) + emean ** 2 * rstd ** 2  # relative
    h = d * rstd
    eh = rstd * emean + h.abs() * (ers + 3 * E)
    return (emean.reshape(N, G), (rstd * ers).reshape(N, G), eh.reshape(N, L, C), h.reshape(N, L, C),
            ers.expand(N, L, G, C // G).reshape(N, L, C), rstd.expand(N, L, G, C // G).reshape(N, L, C))
