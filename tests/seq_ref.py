"""References of the sequence operators in 64 bits, from the formulas of
include/tg_sequence.h, with bounds on what fp32 arithmetic may be off.

Every function works on CPU float64 tensors of one sequence ([L, C] rows) and
returns (value, bound) pairs. The bounds are first-order rounding analyses:
E = 2^-24 (half a step of fp32) times the number of roundings on the way times
the magnitudes that are rounded. An output held in fewer bits adds half a step
of its type relative to the value (``tol``). Hardware exp2, reciprocal and
square root are counted as one unit in the last place (2 E). Where the exponential's
argument u is rounded n times, the result is off by n*E*|u| relative.
"""
from __future__ import annotations

import torch

E = 2.0 ** -24
F64 = torch.float64


def tol(value, bound, dtype):
    """What an output of ``dtype`` may be off: its rounding of a value that is
    itself off by ``bound``, and half the smallest step near zero."""
    f = torch.finfo(dtype)
    return bound * (1 + f.eps) + (value.abs() + bound) * (f.eps / 2) + f.smallest_normal * f.eps


def check(name, got, want, bound):
    """Every element within its bound, and no NaN where there is none."""
    g = got.detach().double().cpu()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    bad = ~((g - want).abs() <= tol(want, bound, got.dtype))
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d off; first at %s: got %r, want %r within %.3g"
                             % (name, int(bad.sum()), bad.numel(), i, float(g[i]), float(want[i]),
                                float(tol(want, bound, got.dtype)[i])))


# ---- layer norm

def norm_sums(C):
    """Roundings of a sum over a row: at most C in a thread's chain (64, or
    C/1024 for long rows), 6 steps over a wave and 16 over the waves."""
    return max(64, C // 1024 + 1) + 22


def norm(s, gamma, beta, eps):
    """y, mean, rstd of rows s [R, C]; also xhat and the bounds' ingredients."""
    C = s.shape[-1]
    n = norm_sums(C)
    mean = s.mean(-1, keepdim=True)
    d = s - mean
    rstd = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    h = d * rstd
    emean = (n + 2) * E * s.abs().mean(-1, keepdim=True)
    ers = (n + 12) * E  # relative: half of the variance's, the root and the division
    eh = rstd * emean + h.abs() * (ers + 3 * E)
    b = torch.zeros(C, dtype=F64) if beta is None else beta
    y = h * gamma + b
    ey = gamma.abs() * eh + 2 * E * ((h * gamma).abs() + b.abs())
    # A shift of the mean changes the variance to second order only.
    return dict(y=(y, ey), mean=(mean.squeeze(-1), emean.squeeze(-1)),
                rstd=(rstd.squeeze(-1), rstd.squeeze(-1) * ers + rstd.squeeze(-1) ** 3 * (emean.squeeze(-1)) ** 2),
                h=(h, eh), r=rstd)


def norm_grads(dy, s, gamma, eps, dsum=None):
    R, C = s.shape
    f = norm(s, gamma, None, eps)
    h, eh = f["h"]
    n = norm_sums(C)
    g = dy * gamma
    eg = E * g.abs()
    m1, m2 = g.mean(-1, keepdim=True), (g * h).mean(-1, keepdim=True)
    em1 = eg.mean(-1, keepdim=True) + (n + 2) * E * g.abs().mean(-1, keepdim=True)
    em2 = ((g.abs() * eh).mean(-1, keepdim=True) + eg.mul(h.abs()).mean(-1, keepdim=True)
           + (n + 2) * E * (g * h).abs().mean(-1, keepdim=True))
    inner = g - m1 - h * m2
    ein = (eg + em1 + h.abs() * em2 + eh * m2.abs()
           + 3 * E * (g.abs() + m1.abs() + (h * m2).abs()))
    dx = f["r"] * inner
    edx = f["r"] * (ein + (n + 14) * E * inner.abs())
    if dsum is not None:
        dx = dx + dsum
        edx = edx + E * dx.abs()
    dgamma = (dy * h).sum(0)
    edgamma = (dy.abs() * eh).sum(0) + (R + 2) * E * (dy * h).abs().sum(0)
    dbeta = dy.sum(0)
    return dict(dx=(dx, edx), dgamma=(dgamma, edgamma), dbeta=(dbeta, R * E * dy.abs().sum(0)))


# ---- activations

def silu(v, ev):
    """silu and its bound: the argument's error (slope at most 1.1), the
    exponential of -v (argument rounded once), reciprocal and products."""
    y = v * torch.sigmoid(v)
    return y, 1.1 * ev + y.abs() * E * (8 + 2 * v.abs())


def silu_slope(v, ev):
    sg = torch.sigmoid(v)
    d = sg * (1 + v * (1 - sg))
    # sigmoid is off by (2|v| + 6) E relative, 1 - sigmoid by that absolute.
    es = sg * E * (6 + 2 * v.abs())
    return d, 0.5 * ev + es * (1 + 2 * v.abs()) + 4 * E * (sg * (1 + v.abs()))


# ---- short causal convolution

def _windows(x, init, K):
    rows = torch.cat([init, x]) if K > 1 else x
    return torch.stack([rows[k:k + x.shape[0]] for k in range(K)])  # [K, L, D]


def conv(x, w, bias, act, init):
    """(y, bound), last K-1 rows."""
    K, D = w.shape
    win = _windows(x, init, K)
    b = torch.zeros(D, dtype=F64) if bias is None else bias
    v = b + (w[:, None] * win).sum(0)
    ev = (K + 1) * E * (b.abs() + (w[:, None] * win).abs().sum(0))
    rows = torch.cat([init, x])
    last = rows[rows.shape[0] - (K - 1):]
    return (silu(v, ev) if act else (v, ev)), last, (v, ev, win)


def conv_grads(dy, x, w, bias, act, init, dlast=None):
    K, D = w.shape
    L = x.shape[0]
    _, _, (v, ev, win) = conv(x, w, bias, act, init)
    if act:
        sl, esl = silu_slope(v, ev)
        g, eg = dy * sl, dy.abs() * esl + E * (dy * sl).abs()
    else:
        g, eg = dy, torch.zeros_like(dy)
    rows = torch.zeros(L + K - 1, D, dtype=F64)
    erows = torch.zeros_like(rows)
    for k in range(K):
        rows[k:k + L] += w[k] * g
        erows[k:k + L] += w[k].abs() * (eg + (K + 1) * E * g.abs())
    if dlast is not None:
        rows[L:] += dlast
        erows[L:] += E * rows[L:].abs()
    dw = (g * win).sum(1)
    edw = (eg * win.abs()).sum(1) + (L + 2) * E * (g * win).abs().sum(1)
    return dict(dx=(rows[K - 1:], erows[K - 1:]), dinit=(rows[:K - 1], erows[:K - 1]),
                dw=(dw, edw), dbias=(g.sum(0), eg.sum(0) + (L + 2) * E * g.abs().sum(0)))


# ---- selective scan

def softplus(v):
    """Value and bound: exp(-|v|) rounded argument, log1p to 3 units, one sum;
    near v = 0 the argument's own rounding enters with slope 1/2."""
    d = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    return d, d * E * (10 + 2 * torch.clamp(-v, min=0))


def _spread(m, D):
    """[L, G, N] -> [L, D, N]."""
    L, G, N = m.shape
    return m.reshape(L, G, 1, N).expand(L, G, D // G, N).reshape(L, D, N)


def scan(x, dt, A, B, C, skip, z, bias, use_softplus, init):
    """y, final state, and everything the gradients need. B, C: [L, G, N].

    h is off by eh: each step's decay by its own rounding and its argument's
    (d and d*A: c), the input by three roundings. Splitting the steps and
    joining the parts rounds no more often than stepping does; the doubled
    count (2 *) covers both."""
    L, D = x.shape
    N = A.shape[1]
    raw = dt + (bias if bias is not None else 0.0)
    eraw = E * raw.abs()
    if use_softplus:
        d, ed = softplus(raw)
        ed = ed + torch.sigmoid(raw) * eraw
    else:
        d, ed = raw, eraw
    Bs, Cs = _spread(B, D), _spread(C, D)
    a = torch.exp(d[..., None] * A)
    arg = (d[..., None] * A).abs()
    ea = 2 * a * (3 * E + 4 * E * arg + ed[..., None] * A.abs())
    u = d * x
    eu = ed * x.abs() + E * u.abs()
    b = u[..., None] * Bs
    eb = eu[..., None] * Bs.abs() + 2 * E * b.abs()
    hs, ehs, h, H, eh = [], [], init, init.abs(), torch.zeros_like(init)
    for t in range(L):
        eh = a[t] * eh + ea[t] * H + eb[t] + 2 * E * (a[t] * H + b[t].abs())
        H = a[t] * H + b[t].abs()
        h = a[t] * h + b[t]
        hs.append(h)
        ehs.append(eh)
    hs = torch.stack(hs) if L else torch.zeros(0, D, N, dtype=F64)
    ehs = torch.stack(ehs) if L else torch.zeros(0, D, N, dtype=F64)
    sk = skip if skip is not None else torch.zeros(D, dtype=F64)
    v = (hs * Cs).sum(-1) + sk * x
    ev = (ehs * Cs.abs()).sum(-1) + (N + 4) * E * ((hs * Cs).abs().sum(-1) + (sk * x).abs())
    if z is not None:
        gz, egz = silu(z, torch.zeros_like(z))
        y = (v * gz, ev * gz.abs() + v.abs() * egz + E * (v * gz).abs())
    else:
        y = (v, ev)
    keep = dict(raw=raw, eraw=eraw, d=d, ed=ed, a=a, ea=ea, u=u, eu=eu, hs=hs, ehs=ehs, v=v, ev=ev,
                Bs=Bs, Cs=Cs, sk=sk)
    return y, (h, eh), keep


def scan_grads(dy, x, dt, A, B, C, skip, z, bias, use_softplus, init, dfinal=None):
    L, D = x.shape
    N, G = A.shape[1], B.shape[1]
    _, _, k = scan(x, dt, A, B, C, skip, z, bias, use_softplus, init)
    out = {}
    if z is not None:
        zero = torch.zeros_like(z)
        gz, egz = silu(z, zero)
        sl, esl = silu_slope(z, zero)
        dv, edv = dy * gz, dy.abs() * egz + E * (dy * gz).abs()
        out["dz"] = (dy * k["v"] * sl, dy.abs() * (k["ev"] * sl.abs() + k["v"].abs() * esl)
                     + 3 * E * (dy * k["v"] * sl).abs())
    else:
        dv, edv = dy, torch.zeros_like(dy)
    a, ea, hs, ehs = k["a"], k["ea"], k["hs"], k["ehs"]
    carry = torch.zeros(D, N, dtype=F64) if dfinal is None else dfinal
    ecarry = torch.zeros_like(carry)
    M = carry.abs()
    r = dict(ddt=[], eddt=[], dx=[], edx=[], dB=[], edB=[], dC=[], edC=[])
    dA, edA = torch.zeros(D, N, dtype=F64), torch.zeros(D, N, dtype=F64)
    for t in range(L - 1, -1, -1):
        Bt, Ct = k["Bs"][t], k["Cs"][t]
        d, ed, u, eu = k["d"][t][:, None], k["ed"][t][:, None], k["u"][t][:, None], k["eu"][t][:, None]
        g = dv[t][:, None] * Ct + carry
        Mg = (dv[t][:, None] * Ct).abs() + M
        eg = edv[t][:, None] * Ct.abs() + ecarry + 2 * E * Mg
        hp = hs[t - 1] if t else init
        ehp = ehs[t - 1] if t else torch.zeros_like(init)
        w = g * a[t] * hp  # dL/d(log a)
        ew = eg * a[t] * hp.abs() + Mg * (ea[t] * hp.abs() + a[t] * ehp) + 3 * E * Mg * a[t] * hp.abs()
        f1, ef1 = (w * A).sum(-1), (ew * A.abs()).sum(-1) + (N + 6) * E * (w * A).abs().sum(-1)
        f2, ef2 = (g * Bt).sum(-1), (eg * Bt.abs()).sum(-1) + (N + 4) * E * (g * Bt).abs().sum(-1)
        xt = x[t]
        dd = f1 + f2 * xt
        edd = ef1 + ef2 * xt.abs() + 2 * E * (f1.abs() + (f2 * xt).abs())
        if use_softplus:
            sg = torch.sigmoid(k["raw"][t])
            esg = sg * E * (6 + 2 * k["raw"][t].abs()) + 0.25 * k["eraw"][t]
            dd, edd = dd * sg, edd * sg + dd.abs() * esg + E * (dd * sg).abs()
        r["ddt"].append(dd), r["eddt"].append(edd)
        dx = d[:, 0] * f2 + k["sk"] * dv[t]
        r["dx"].append(dx)
        r["edx"].append(d[:, 0] * ef2 + ed[:, 0] * f2.abs() + k["sk"].abs() * edv[t]
                        + 3 * E * ((d[:, 0] * f2).abs() + (k["sk"] * dv[t]).abs()))
        gu, egu = g * u, eg * u.abs() + Mg * eu + E * (g * u).abs()
        dh, edh = dv[t][:, None] * hs[t], edv[t][:, None] * hs[t].abs() + dv[t][:, None].abs() * ehs[t]
        for name, val, err in (("dB", gu, egu), ("dC", dh, edh)):
            val, err = val.reshape(G, D // G, N), err.reshape(G, D // G, N)
            r[name].append(val.sum(1))
            r["e" + name].append(err.sum(1) + (D // G + 4) * E * val.abs().sum(1))
        dA = dA + w * d
        edA = edA + ew * d.abs() + (w * ed).abs() + (L + 4) * E * (w * d).abs()
        ecarry = eg * a[t] + Mg * ea[t] + E * Mg * a[t]
        M = Mg * a[t]
        carry = g * a[t]
    for name, width in (("ddt", (D,)), ("dx", (D,)), ("dB", (G, N)), ("dC", (G, N))):
        stack = lambda v: torch.stack(v[::-1]) if v else torch.zeros((0,) + width, dtype=F64)  # noqa: E731
        out[name] = (stack(r[name]), stack(r["e" + name]))
    out["dA"] = (dA, edA)
    out["dD"] = ((dv * x).sum(0), (edv * x.abs()).sum(0) + (L + 2) * E * (dv * x).abs().sum(0))
    ddt, eddt = out["ddt"]
    out["dbias"] = (ddt.sum(0), eddt.sum(0) + (L + 2) * E * ddt.abs().sum(0))
    out["dinit"] = (carry, ecarry)
    return out
