"""The 64-bit references of the sequence operators (tests/seq_ref.py) by
themselves, on the CPU: forward passes against straightforward loops, and the
gradient formulas against central differences of the forward passes. One
mistake planted in each formula must show."""
import pytest
import torch

import seq_ref as R

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=F64)


def _difference(loss, t, direction, step=1e-5):
    """Derivative of loss() along ``direction`` of t (changed in place)."""
    t += step * direction
    up = loss()
    t -= 2 * step * direction
    down = loss()
    t += step * direction
    return (up - down) / (2 * step)


def _assert_gradient(loss, pairs):
    for i, (name, t, grad) in enumerate(pairs):
        if t.numel() == 0:
            continue
        u = _rand(*t.shape, seed=100 + i)
        want = float(_difference(loss, t, u))
        got = float((grad * u).sum())
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), (name, got, want)


def _assert_not_gradient(loss, t, grad):
    u = _rand(*t.shape, seed=100)
    want = float(_difference(loss, t, u))
    assert abs(float((grad * u).sum()) - want) > 1e-6 * (1 + abs(want))


@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (5, 17)])
def test_norm_gradients(shape):
    s, gamma, beta, dy, ds = (_rand(*sh, seed=i) for i, sh in
                              enumerate((shape, shape[1:], shape[1:], shape, shape)))
    loss = lambda: (R.norm(s, gamma, beta, 1e-5)["y"][0] * dy).sum() + (s * ds).sum()  # noqa: E731
    g = R.norm_grads(dy, s, gamma, 1e-5, ds)
    _assert_gradient(loss, [("dx", s, g["dx"][0]), ("dgamma", gamma, g["dgamma"][0]),
                            ("dbeta", beta, g["dbeta"][0])])
    if shape[1] > 2:
        _assert_not_gradient(loss, s, g["dx"][0] + R.norm(s, gamma, None, 1e-5)["h"][0] * 1e-3)


@pytest.mark.parametrize("L,K,act", [(0, 4, True), (1, 4, True), (2, 2, False), (7, 3, True), (9, 8, True)])
def test_conv_gradients(L, K, act):
    D = 3
    x, w, bias, init = _rand(L, D), _rand(K, D), _rand(D), _rand(K - 1, D, seed=9)
    dy, dlast = _rand(L, D, seed=5), _rand(K - 1, D, seed=6)

    def loss():
        (y, _), last, _ = R.conv(x, w, bias, act, init)
        return (y * dy).sum() + (last * dlast).sum()
    # the forward pass itself, token by token
    (y, _), last, _ = R.conv(x, w, bias, act, init)
    rows = torch.cat([init, x])
    for t in range(L):
        v = bias + sum(w[k] * rows[t + k] for k in range(K))
        assert torch.allclose(y[t], v * torch.sigmoid(v) if act else v)
    assert torch.equal(last, rows[L:])
    g = R.conv_grads(dy, x, w, bias, act, init, dlast)
    _assert_gradient(loss, [("dx", x, g["dx"][0]), ("dw", w, g["dw"][0]),
                            ("dbias", bias, g["dbias"][0]), ("dinit", init, g["dinit"][0])])
    if L > 1:
        _assert_not_gradient(loss, w, g["dw"][0].roll(1, 0))


@pytest.mark.parametrize("L,G,gate,soft", [(0, 1, True, True), (1, 1, True, True), (6, 2, True, True),
                                           (9, 1, False, True), (5, 2, True, False)])
def test_scan_gradients(L, G, gate, soft):
    D, N = 4, 3
    x, dt, skip, bias = _rand(L, D), _rand(L, D, seed=1), _rand(D), _rand(D, seed=2)
    if not soft:
        dt, bias = dt.abs() * 0.1, bias.abs() * 0.1
    A, B, C = -_rand(D, N).abs() - 0.1, _rand(L, G, N, seed=3), _rand(L, G, N, seed=4)
    z = _rand(L, D, seed=5) if gate else None
    init, dy, dfinal = _rand(D, N, seed=6), _rand(L, D, seed=7), _rand(D, N, seed=8)

    def loss():
        (y, _), (h, _), _ = R.scan(x, dt, A, B, C, skip, z, bias, soft, init)
        return (y * dy).sum() + (h * dfinal).sum()
    g = R.scan_grads(dy, x, dt, A, B, C, skip, z, bias, soft, init, dfinal)
    pairs = [("dx", x, g["dx"][0]), ("ddt", dt, g["ddt"][0]), ("dA", A, g["dA"][0]),
             ("dB", B, g["dB"][0]), ("dC", C, g["dC"][0]), ("dD", skip, g["dD"][0]),
             ("dbias", bias, g["dbias"][0]), ("dinit", init, g["dinit"][0])]
    if gate:
        pairs.append(("dz", z, g["dz"][0]))
    _assert_gradient(loss, pairs)
    if L > 1:
        _assert_not_gradient(loss, dt, g["ddt"][0] + 1e-3 * g["dx"][0])


def test_softplus_small_and_large():
    v = torch.tensor([-80.0, -20.0, -5.0, 0.0, 3.0, 40.0], dtype=F64)
    d, b = R.softplus(v)
    assert torch.allclose(d, torch.nn.functional.softplus(v, threshold=1e9), rtol=1e-12)
    assert bool((b > 0).all())


def test_check_reports_a_wrong_value():
    want = torch.ones(3, dtype=F64)
    R.check("fine", torch.ones(3), want, torch.zeros(3, dtype=F64))
    with pytest.raises(AssertionError, match="wrong"):
        R.check("wrong", torch.tensor([1.0, 1.001, 1.0]), want, torch.zeros(3, dtype=F64))
    with pytest.raises(AssertionError, match="nan"):
        R.check("nan", torch.tensor([1.0, float("nan"), 1.0]), want, torch.zeros(3, dtype=F64))
