"""Group norm at the ends of its range: means far past the root of fp32's largest
number, against the bounds of delta_ref.py."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import delta_ref as D
import seq_ref as R
from gpu_cases import note
from test_group_norm_gpu import BF16, F32, Case, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# Maps of one chunk and of many, whole groups in a vector and across vectors, odd
# channels, a long group of single rows, heads.
SHAPES = [((2, 60, 16), 4), ((1, 5000, 8), 2), ((2, 9, 33), 3), ((3, 700), 1), ((2, 3, 4104), 2), ((5, 64), 4)]


@pytest.mark.parametrize("shape,G", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("value", [3e19, -3e19, 1e30, -1e35])
def test_constant_groups_of_any_size(shape, G, dtype, value):
    """No spread: the result is beta, the mean the value (its sum within fp32)."""
    note("group norm of %g %s %s" % (value, shape, dtype))
    C = shape[-1]
    x = torch.full(shape, value, dtype=dtype, device="cuda")
    gamma, beta = torch.ones(C, device="cuda"), torch.linspace(-1, 1, C, device="cuda")
    y, mean, rstd = tg.group_norm_train(x, G, gamma, beta, act="none")
    assert torch.equal(y, beta.to(dtype).expand(shape))
    assert torch.equal(mean, x.float().reshape(shape[0], -1)[:, :1].expand_as(mean))
    assert torch.equal(rstd, torch.full_like(rstd, float(rstd[0, 0]))) and abs(float(rstd[0, 0]) * 1e-5 ** 0.5 - 1) < 1e-6
    d = tg.group_norm_backward(torch.ones_like(x), x, G, gamma, mean, rstd, beta, act="none")
    assert not d.dgamma.any() and bool(torch.isfinite(d.dx).all()) and bool(torch.isfinite(d.dbeta).all())


@pytest.mark.parametrize("shape,G", SHAPES, ids=str)
def test_means_past_the_root_of_the_largest_number(shape, G):
    """A mean of 1e20 with a spread of 1e16: every element within its bound."""
    c = Case((shape, G, "f32", "none", True, False, 0))
    c.x = c.x * 1e16 + 1e20
    want, mean, rstd = D.group_norm(c.flat(c.x), G, c.gamma.double(), c.beta.double(), 1e-5, "none", None)
    b = c.bounds()
    y, m, r = tg.group_norm_train(*c.args(), **c.more())
    R.check("y", y, want.reshape(shape), b["y"][1].reshape(shape))
    R.check("mean", m, mean, b["mean"])
    R.check("rstd", r, rstd, b["rstd"])


@pytest.mark.parametrize("shape,G", [((1, 20, 256), 256), ((2, 60, 16), 4), ((3, 700), 1)], ids=str)
def test_a_spread_past_fp32_is_not_taken_for_none(shape, G):
    """Squares that are infinite: y is what it should be, or no number, or nothing of h
    is left (a variance of infinity), but never a multiple of x."""
    c = Case((shape, G, "f32", "none", False, False, 0))
    c.x = c.x * 1e20
    want, _, _ = D.group_norm(c.flat(c.x), c.G, c.gamma.double(), None, 1e-5, "none", None)
    y = tg.group_norm(*c.args(), **c.more()).double().cpu().reshape(want.shape)
    assert bool((torch.isnan(y) | (y.abs() <= 1.01 * want.abs())).all())


def sums_of(c, mean, rstd, got):
    """gamma's and beta's gradients against their sums in 64 bits."""
    shape, G, C = c.shape, c.G, c.shape[-1]
    leaf = [c.gamma.double().requires_grad_(), c.beta.double().requires_grad_()]
    x64, dy64, z64 = c.flat(c.x), c.flat(c.dy), c.flat(c.z)
    out, _, _ = D.group_norm(x64, G, leaf[0], leaf[1], 1e-5, "silu", z64)
    want = torch.autograd.grad((out * dy64).sum(), leaf)
    h = ((x64.reshape(shape[0], -1, G, C // G) - mean.double().cpu()[:, None, :, None])
         * rstd.double().cpu()[:, None, :, None]).reshape(x64.shape)
    v = h * c.gamma.double() + c.beta.double()
    s = torch.sigmoid(v)
    dv = dy64 * (1 if z64 is None else z64 * torch.sigmoid(z64)) * s * (1 + v * (1 - s))
    rows = dv.shape[0] * dv.shape[1]
    # Single roundings: of h (the mean's among them), v, the slopes, products: of each term.
    for name, w, terms in (("dgamma", want[0], dv * h), ("dbeta", want[1], dv)):
        big = (dy64.abs() * (1 if z64 is None else z64.abs()) * (1 + h.abs()) ** 2 * (1 + c.gamma.abs().max()))
        bound = 32 * D.E * big.sum((0, 1)) + (rows + 64) ** 0.5 * 8 * D.E * terms.abs().sum((0, 1))
        bad = ~((getattr(got, name).double().cpu() - w).abs() <= bound)
        assert not bad.any(), (name, int(bad.sum()))


# Maps and long groups by the thousand, the first of them more than the backward pass
# holds channels' sums of at once.
MANY = [((4500, 4120), 1, BF16), ((2500, 1, 600), 2, F32), ((3001, 700), 1, BF16), ((2100, 3, 40), 4, F32), ((5000, 2, 2, 33), 3, BF16)]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape,G,dtype", MANY, ids=str)
def test_many_maps(shape, G, dtype, gate):
    """Gradients of all, against the same maps a few at a time; gamma's and beta's
    against their sum in 64 bits."""
    note("group norm, many maps %s %s %s" % (shape, dtype, gate))
    c = Case((shape, G, "f32" if dtype is F32 else "bf16", "silu", True, gate, 0))
    (x, _, gamma), more, dy = c.args(), c.more(), up(c.dy)
    z = more.pop("z")
    y, mean, rstd = tg.group_norm_train(x, G, gamma, z=z, **more)
    got = tg.group_norm_backward(dy, x, G, gamma, mean, rstd, z=z, **more)
    again = tg.group_norm_backward(dy, x, G, gamma, mean, rstd, z=z, **more)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    for lo in range(0, shape[0], 500):
        cut = lambda t: None if t is None else t[lo:lo + 500]  # noqa: E731
        some = tg.group_norm_backward(cut(dy), cut(x), G, gamma, cut(mean), cut(rstd), z=cut(z), **more)
        assert torch.equal(some.dx, got.dx[lo:lo + 500])
        assert z is None or torch.equal(some.dz, got.dz[lo:lo + 500])
    sums_of(c, mean, rstd, got)


# More rows than the heads kernel has in flight (512 backward, 2048 * 2048 / C forward), the
# last round for some of a wave's rows only; groups of one lane, of a wave, across vectors.
ROUNDS = [((1100, 64), 4, "bf16"), ((1999, 24), 3, "f32"), ((1301, 33), 3, "f16"), ((2500, 2048), 16, "bf16"), ((2300, 2048), 8, "f32"),
          ((1030, 512), 2, "f16"), ((530, 16), 1, "f32"), ((2700, 100), 50, "bf16")]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape,G,dt", ROUNDS, ids=str)
def test_many_rows_of_heads(shape, G, dt, gate):
    """Forward and backward against calls of fewer rows than are in flight, which
    test_group_norm_gpu.py holds against 64 bits; gamma's and beta's gradients here."""
    note("group norm, many rows %s %s %s" % (shape, dt, gate))
    c = Case((shape, G, dt, "silu", True, gate, 0))
    (x, _, gamma), more, dy = c.args(), c.more(), up(c.dy)
    z = more.pop("z")
    y, mean, rstd = tg.group_norm_train(x, G, gamma, z=z, **more)
    assert torch.equal(y, tg.group_norm(x, G, gamma, z=z, **more))
    got = tg.group_norm_backward(dy, x, G, gamma, mean, rstd, z=z, **more)
    for lo in range(0, shape[0], 300):
        cut = lambda t: None if t is None else t[lo:lo + 300]  # noqa: E731
        some = tg.group_norm_train(cut(x), G, gamma, z=cut(z), **more)
        assert all(torch.equal(a, b[lo:lo + 300]) for a, b in zip(some, (y, mean, rstd)))
        d = tg.group_norm_backward(cut(dy), cut(x), G, gamma, cut(mean), cut(rstd), z=cut(z), **more)
        assert torch.equal(d.dx, got.dx[lo:lo + 300])
        assert z is None or torch.equal(d.dz, got.dz[lo:lo + 300])
    sums_of(c, mean, rstd, got)
