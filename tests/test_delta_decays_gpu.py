"""Gradients of the gated delta rule's decays where decays are strong: every term of a
token's gradient carries that token's own decay, so a strong decay leaves a small
gradient, and none where the decay is taken as 0."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import delta_ref as D
from gpu_cases import note
from test_delta_gpu import F32, TYPES, Case, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def strong(case, seed=0):
    """Plain gates; decays of e^-0.01 to e^-200 among ones near 1, rates of three sizes."""
    c = Case(case, seed)
    g = torch.Generator().manual_seed(seed + 11)
    step = torch.rand(c.T, c.HV, generator=g) * 0.01
    step[::7] = 0.0
    step[5::11] += torch.rand(step[5::11].shape, generator=g) * 2.0
    c.dt = step.to(c.dtype)
    c.A = torch.tensor([-1.0, -30.0, -1e5])[:c.HV]
    return c


def want(c):
    """The decays' gradients dg [T, HV] and the size of what each is a sum of."""
    q, k, v, dt, A, beta = (t.double() for t in (c.q, c.k, c.v, c.dt, c.A, c.beta))
    _, g, b = D.gates(dt, A, beta, None, False, False)
    q, k = D.spread(q, c.HV), D.spread(k, c.HV)
    total, held = 0, []
    for i, (lo, hi) in enumerate(zip(c.bounds[:-1], c.bounds[1:])):
        S = c.initial[i].double().requires_grad_()
        for t in range(lo, hi):
            S = torch.exp(g[t])[:, None, None] * S
            S.retain_grad()
            held.append(S)
            u = b[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
            S = S + k[t][:, :, None] * u[:, None, :]
            total = total + (0.7 * torch.einsum("hk,hkv->hv", q[t], S) * c.dy[t].double()).sum()
        total = total + (S * c.dstate[i].double()).sum()
    total.backward()
    dg = torch.stack([(S.grad * S.detach()).sum((1, 2)) for S in held])
    size = torch.stack([S.grad.flatten(1).norm(dim=1) * S.detach().flatten(1).norm(dim=1) for S in held])
    kap = max(D.kappa(k[lo:hi], g[lo:hi], b[lo:hi], 64) for lo, hi in zip(c.bounds[:-1], c.bounds[1:]) if hi > lo)
    return g, dg, size, kap


STRONG = [([100], False, 1, 3, 16, 8, "f32", True, True, 0), ([130, 3, 0, 70], True, 1, 3, 40, 24, "f32", True, True, 0),
          ([150], False, 3, 3, 64, 32, "bf16", True, True, 0), ([90], False, 1, 3, 32, 16, "f16", True, True, 0),
          ([60], False, 1, 2, 200, 16, "f32", True, True, 0), ([1400], False, 1, 1, 16, 16, "f32", True, True, 0),
          ([1400], False, 1, 3, 16, 16, "f32", True, True, 0)]


@pytest.mark.parametrize("case", STRONG, ids=str)
def test_every_token_of_strong_decays(case):
    """A decay's logarithm g has few roundings, which its exponential makes 4 E |g| of
    the result; those of other tokens on the way at most as much as x e^-x <= 1."""
    note("delta strong decays %s" % (case,))
    c = strong(case)
    g, dg, size, kap = want(c)
    chunks = max(-(-n // 32) for n in c.lengths)
    _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **c.more())
    A = c.A.double()
    ddt, out = dg * A, got.ddt.double().cpu().reshape(dg.shape)
    rel = D.allowed(F32, kap, chunks, gradient=True) + 4 * D.E * (g.abs() + 1)
    # Decays below 2^-126 are taken as 0.
    bound = rel * size * A.abs() + (torch.finfo(c.dtype).eps / 2) * ddt.abs() + 1e-30
    bound = bound + torch.finfo(c.dtype).smallest_normal * torch.finfo(c.dtype).eps
    past = ddt.abs() - bound > torch.finfo(c.dtype).max
    bad = ~((out - ddt).abs() <= bound) & ~(past & torch.isinf(out))
    assert not bad.any(), [(i.tolist(), float(out[tuple(i)]), float(ddt[tuple(i)]), float(bound[tuple(i)]))
                           for i in bad.nonzero()[:4]]
    gone = g < -100
    assert not out[gone].any() and (c.HV < 3 or bool(gone.any()))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("plain", [False, True])
def test_infinite_rates_have_no_gradient(dt, plain):
    """Gradients as with a rate that is merely enormous, and none of the rate itself or
    of its steps, also where a step of zero keeps the state."""
    c = Case(([100], False, 1, 3, 32, 16, dt, True, plain, 0))
    if plain:
        c.dt[3::9] = 0.0
    c.A = torch.tensor([-0.5, -float("inf"), -1.0])
    big = torch.tensor([-0.5, -1e30, -1.0])

    def run(A):
        c.A = A
        _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
        return tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **c.more())
    a, b = run(c.A), run(big)
    for name in ("dq", "dk", "dv", "dbeta", "dinitial_state"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert not a.ddt[..., 1].any() and float(a.dA[1]) == 0
    assert torch.equal(a.ddt[..., ::2], b.ddt[..., ::2]) and torch.equal(a.dA[::2], b.dA[::2])
    if not plain:
        assert float(a.ddt_bias[1]) == 0 and torch.equal(a.ddt_bias[::2], b.ddt_bias[::2])


def test_infinite_steps():
    """They forget the state like any decay that is taken as 0."""
    c = Case(([70], False, 1, 2, 16, 8, "f32", True, False, 0))
    c.dt[20] = float("inf")
    _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **c.more())
    assert not got.ddt[0, 20].any() and all(bool(torch.isfinite(t).all()) for t in got)


@pytest.mark.parametrize("lengths", [[300], [65, 200, 1], [1500]], ids=str)
def test_gradients_of_growing_decays(lengths):
    """Decays above 1: a share u of the largest state, or of its gradient, grows by no
    more than all decays together on its way, so that the product of both may be off by
    e^2G times what it may be off without growth."""
    c = Case((lengths, True, 1, 2, 16, 24, "f32", True, False, 0))
    c.dt_bias, c.A = None, torch.tensor([1.0, 0.5])
    c.dt = torch.full((c.T, 2), 1.5 / max(lengths))
    leaf = [t.double().requires_grad_() for t in (c.q, c.k, c.v, c.dt, c.A, c.beta, c.initial)]
    q, k, v, dt, A, beta, initial = leaf
    y, state, _, kap, chunks = D.delta(c.bounds, q, k, v, dt, A, beta, None, False, True, True, None, initial)
    want = torch.autograd.grad((y * c.dy.double()).sum() + (state * c.dstate.double()).sum(), leaf)
    more = dict(initial_state=up(c.initial), offsets=c.offsets, softplus=False)
    _, saved = tg.gated_delta_rule_train(*c.args(), **more)
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **more)
    allowed = 2 * (2 * chunks * D.STEPS) ** 0.5 * kap * kap * D.E * float(torch.exp(torch.tensor(2 * 1.5)))
    for name, w in zip(("dq", "dk", "dv", "ddt", "dA", "dbeta", "dinitial_state"), want):
        d = float((getattr(got, name).double().cpu().reshape(w.shape) - w).norm() / w.norm())
        assert d <= allowed, "%s: %.3g, allowed %.3g" % (name, d, allowed)
