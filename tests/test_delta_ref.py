"""The 64-bit references of delta_ref.py against central differences of their own
values: the gradients that the GPU tests take from automatic differentiation are
those of the formulas."""
from __future__ import annotations

import torch

import delta_ref as D

F64 = torch.float64


def _differences(f, leaf, weights, step=1e-6):
    out = torch.zeros_like(leaf)
    flat, o = leaf.view(-1), out.view(-1)
    for i in range(flat.numel()):
        x = float(flat[i])
        flat[i] = x + step
        up = float((f() * weights).sum())
        flat[i] = x - step
        o[i] = (up - float((f() * weights).sum())) / (2 * step)
        flat[i] = x
    return out


def test_delta_gradients():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    leaves = dict(q=r(6, 1, 3), k=r(6, 1, 3), v=r(6, 2, 2), dt=r(6, 2), A=-r(2).abs(), beta=r(6, 2), dt_bias=r(2),
                  initial=r(2, 2, 3, 2))
    weights = r(6, 2, 2)
    call = lambda: D.delta([0, 4, 6], **leaves)[0]  # noqa: E731
    for t in leaves.values():
        t.requires_grad_()
    want = torch.autograd.grad((call() * weights).sum(), list(leaves.values()))
    with torch.no_grad():
        for (name, t), w in zip(leaves.items(), want):
            near = _differences(call, t, weights)
            assert float((near - w).abs().max()) < 1e-7 * max(1.0, float(w.abs().max())), name


def test_group_norm_gradients():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    x, gamma, beta, z, w = r(2, 3, 4), r(4), r(4), r(2, 3, 4), r(2, 3, 4)
    for act in ("silu", "none"):
        call = lambda: D.group_norm(x, 2, gamma, beta, 1e-5, act, z)[0]  # noqa: E731
        leaves = [t.requires_grad_() for t in (x, gamma, beta, z)]
        want = torch.autograd.grad((call() * w).sum(), leaves)
        with torch.no_grad():
            for t, v in zip(leaves, want):
                assert float((_differences(call, t, w) - v).abs().max()) < 1e-6 * max(1.0, float(v.abs().max()))


def test_delta_of_one_token():
    """By hand: y = scale b (k.q) (v - a k S) + scale a q S."""
    q, k, v = (torch.tensor([[x]], dtype=F64) for x in ([0.6, 0.8], [1.0, 0.0], [2.0]))
    S = torch.tensor([[[[3.0], [5.0]]]], dtype=F64)
    dt, beta = torch.tensor([[0.5]], dtype=F64), torch.tensor([[0.25]], dtype=F64)
    y, state, _, _, _ = D.delta([0, 1], q, k, v, dt, torch.tensor([-2.0], dtype=F64), beta, softplus=False,
                                sigmoid=False, normalize=False, scale=1.0, initial=S)
    a = torch.exp(torch.tensor(-1.0, dtype=F64))
    u = 0.25 * (2 - a * 3)
    assert abs(float(state[0, 0, 0, 0] - (a * 3 + u))) < 1e-15 and abs(float(state[0, 0, 1, 0] - a * 5)) < 1e-15
    assert abs(float(y - (0.6 * (a * 3 + u) + 0.8 * a * 5))) < 1e-14
