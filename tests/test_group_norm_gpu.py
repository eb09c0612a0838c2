"""Group norm on the GPU against the 64-bit reference of delta_ref.py, every element
within bounds of first order in the roundings, for maps, heads of tokens and
groups of every length; gradients against automatic differentiation."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import delta_ref as D
import seq_ref as R
from gpu_cases import note

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = {"f16": F16, "bf16": BF16, "f32": F32}
E = D.E

# shape, groups, type, act, beta, gate, extra row width
CASES = [
    ((1, 1, 1), 1, "f32", "silu", True, False, 0), ((3, 4), 2, "f16", "none", True, True, 0),
    ((2, 5, 7, 12), 3, "f32", "silu", True, False, 0), ((2, 5, 7, 12), 3, "bf16", "silu", False, True, 4),
    ((4, 64), 4, "bf16", "none", True, True, 0), ((5, 96), 2, "f16", "silu", True, False, 8), ((3, 2048), 16, "bf16", "none", True, True, 0),
    ((7, 363), 3, "f32", "silu", True, True, 0), ((2, 600), 2, "f32", "none", True, False, 0), ((2, 3000), 3, "f16", "silu", True, True, 0),
    ((2, 9, 363), 3, "f32", "silu", True, False, 1), ((3, 49, 64), 32, "f16", "silu", True, False, 0), ((1, 33, 17), 17, "bf16", "silu", True, True, 0),
    ((2, 40, 2100), 1, "f16", "silu", True, False, 0), ((1, 5, 4104), 2, "bf16", "none", True, False, 0), ((2, 1000, 24), 4, "f32", "silu", True, True, 0),
    ((1, 7000, 8), 8, "f16", "silu", True, False, 0), ((3, 14, 14, 256), 32, "bf16", "silu", True, False, 0), ((300, 256), 2, "f16", "none", True, True, 0),
    ((2, 3, 9000), 9, "f32", "silu", True, False, 0), ((1, 2, 4096), 4096, "f16", "silu", True, False, 0), ((70, 1, 40), 40, "bf16", "none", False, False, 0),
]


def up(t, wide=0):
    if t is None or not wide:
        return None if t is None else t.cuda()
    big = torch.full(t.shape[:-1] + (t.shape[-1] + wide,), float("nan"), dtype=t.dtype, device="cuda")
    big[..., wide:] = t.cuda()
    return big[..., wide:]


class Case:
    def __init__(self, case, shift=0.4):
        self.shape, self.G, dt, self.act, beta, gate, self.wide = case
        self.dtype, C = TYPES[dt], self.shape[-1]
        g = torch.Generator().manual_seed(sum(self.shape) * 7 + self.G)
        r = lambda *s, scale=1.0, shift=0.0: torch.randn(*s, generator=g) * scale + shift  # noqa: E731
        self.x, self.dy = r(*self.shape, scale=1.5, shift=shift).to(self.dtype), r(*self.shape).to(self.dtype)
        self.z = r(*self.shape).to(self.dtype) if gate else None
        self.gamma, self.beta = r(C, scale=0.3, shift=1.0), r(C, scale=0.3) if beta else None

    def flat(self, t):
        return None if t is None else t.double().reshape(self.shape[0], -1, self.shape[-1])

    def args(self):
        return up(self.x, self.wide), self.G, up(self.gamma)

    def more(self):
        return dict(beta=up(self.beta), act=self.act, z=up(self.z, self.wide))

    def bounds(self):
        """y, its slopes and their bounds, elementwise."""
        x, z = self.flat(self.x), self.flat(self.z)
        b = torch.zeros(self.shape[-1], dtype=torch.float64) if self.beta is None else self.beta.double()
        emean, erstd, eh, h, ers, rstd = D.group_bounds(x, self.G, 1e-5)
        ga = self.gamma.double()
        v = h * ga + b
        ev = ga.abs() * eh + 3 * E * ((h * ga).abs() + b.abs())
        if self.act == "silu":
            a, ea = R.silu(v, ev)
            da, eda = R.silu_slope(v, ev)
        else:
            a, ea, da, eda = v, ev, torch.ones_like(v), torch.zeros_like(v)
        if z is None:
            return dict(y=(a, ea), mean=emean, rstd=erstd, h=(h, eh), da=(da, eda), ers=ers, r=rstd, a=(a, ea), s=None)
        s, es = R.silu(z, torch.zeros_like(z))
        ds, eds = R.silu_slope(z, torch.zeros_like(z))
        return dict(y=(a * s, ea * s.abs() + a.abs() * es + E * (a * s).abs()), mean=emean, rstd=erstd, h=(h, eh), da=(da, eda),
                    ers=ers, r=rstd, a=(a, ea), s=(s, es), ds=(ds, eds))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    note("group norm %s" % (case,))
    c = Case(case)
    b = c.bounds()
    want, mean, rstd = D.group_norm(c.flat(c.x), c.G, c.gamma.double(), c.flat(None) if c.beta is None else c.beta.double(), 1e-5,
                                    c.act, c.flat(c.z))
    y = tg.group_norm(*c.args(), **c.more())
    R.check("y", y, want.reshape(c.shape), b["y"][1].reshape(c.shape))
    y2, m, r = tg.group_norm_train(*c.args(), **c.more())
    assert torch.equal(y, y2)
    R.check("mean", m, mean, b["mean"])
    R.check("rstd", r, rstd, b["rstd"])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    note("group norm backward %s" % (case,))
    c = Case(case)
    leaf = lambda t: None if t is None else t.double().requires_grad_()  # noqa: E731
    x, gamma, beta, z = leaf(c.x), leaf(c.gamma), leaf(c.beta), leaf(c.z)
    N, C = c.shape[0], c.shape[-1]
    flat = lambda t: None if t is None else t.reshape(N, -1, C)  # noqa: E731
    y, _, _ = D.group_norm(flat(x), c.G, gamma, beta, 1e-5, c.act, flat(z))
    leaves = [t for t in (x, gamma, beta, z) if t is not None]
    want = dict(zip([n for n, t in zip(("dx", "dgamma", "dbeta", "dz"), (x, gamma, beta, z)) if t is not None],
                    torch.autograd.grad((y * flat(c.dy.double())).sum(), leaves)))
    _, m, r = tg.group_norm_train(*c.args(), **c.more())
    got = tg.group_norm_backward(up(c.dy, c.wide), *c.args(), m, r, **c.more())
    # dv = dy silu(z) act'(v) and its bound; then the groups' two sums.
    b, dy = c.bounds(), c.flat(c.dy)
    L, G = b["h"][0].shape[1], c.G
    da, eda = b["da"]
    s, es = b["s"] if b["s"] is not None else (torch.ones_like(da), torch.zeros_like(da))
    dv = dy * s * da
    edv = dy.abs() * (s.abs() * eda + es * da.abs()) + 3 * E * dv.abs()
    h, eh = b["h"]
    terms = L * (C // G)
    chain = min(terms, 4096) + 64  # of the longest sum one after another

    def group_mean(t):
        return t.reshape(N, L, G, C // G).mean((1, 3), keepdim=True).expand(N, L, G, C // G).reshape(N, L, C)
    ga = c.gamma.double()
    g, eg = dv * ga, edv * ga.abs() + E * (dv * ga).abs()
    m1, m2 = group_mean(g), group_mean(g * h)
    em1 = group_mean(eg) + chain * E * group_mean(g.abs())
    em2 = group_mean(eg * h.abs() + g.abs() * eh) + chain * E * group_mean((g * h).abs())
    inner = g - m1 - h * m2
    dx, edx = b["r"] * inner, b["r"] * (eg + em1 + h.abs() * em2 + eh * m2.abs() + 4 * E * (g.abs() + m1.abs() + (h * m2).abs())
                                       + b["ers"] * inner.abs())
    R.check("dx", got.dx, want["dx"], edx.reshape(c.shape) + 1e-12 * dx.reshape(c.shape).abs())
    rows = N * L + 64
    eg_ = (dv.abs() * eh + edv * h.abs()).sum((0, 1)) + rows * E * (dv * h).abs().sum((0, 1))
    R.check("dgamma", got.dgamma, want["dgamma"], eg_)
    if c.beta is not None:
        R.check("dbeta", got.dbeta, want["dbeta"], edv.sum((0, 1)) + rows * E * dv.abs().sum((0, 1)))
    if c.z is None:
        assert got.dz is None
    else:
        a, ea = b["a"]
        ds, eds = b["ds"]
        edz = dy.abs() * (ea * ds.abs() + a.abs() * eds) + 4 * E * (dy * a * ds).abs()
        R.check("dz", got.dz, want["dz"], edz.reshape(c.shape))
    again = tg.group_norm_backward(up(c.dy, c.wide), *c.args(), m, r, **c.more())
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, again))


def test_large_mean():
    """A mean a thousand times the spread: the variance must not cancel."""
    for case in (((2, 500, 16), 4, "f32", "none", True, False, 0), ((3, 256), 2, "f32", "none", True, False, 0)):
        c = Case(case, shift=1500.0)
        want, _, _ = D.group_norm(c.flat(c.x), c.G, c.gamma.double(), c.beta.double(), 1e-5, "none", None)
        R.check("y", tg.group_norm(*c.args(), **c.more()), want.reshape(c.shape), c.bounds()["y"][1].reshape(c.shape))


def test_constant_groups_and_outliers():
    """No spread at all, and a first value far from all others."""
    x = torch.full((2, 300, 8), 3.25).cuda()
    g = torch.ones(8).cuda()
    assert not tg.group_norm(x, 2, g, act="none").any()
    x = torch.randn(1, 400, 8, generator=torch.Generator().manual_seed(5)).double()
    x[0, 0, 0] = 3000.0
    want, _, _ = D.group_norm(x.float().double(), 2, torch.ones(8).double(), None, 1e-5, "none", None)
    b = D.group_bounds(x.float().double(), 2, 1e-5)
    R.check("y", tg.group_norm(x.float().cuda(), 2, g, act="none"), want, b[2] + 4 * E * want.abs())


def test_a_bad_value_stays_in_its_group():
    for shape in ((3, 40, 32), (5, 32)):
        c = Case((shape, 4, "f16", "silu", True, True, 0))
        clean = tg.group_norm(*c.args(), **c.more())
        x, G, ga = c.args()
        for bad in (float("nan"), float("inf")):
            t = x.clone()
            t.view(shape[0], -1, 32)[1, 0, 9] = bad
            y = tg.group_norm(t, G, ga, **c.more()).view(shape[0], -1, 4, 8)
            same = clean.view(shape[0], -1, 4, 8)
            mask = torch.ones(shape[0], 4, dtype=torch.bool, device="cuda")
            mask[1, 1] = False
            mask = mask[:, None, :, None].expand_as(y)
            assert torch.equal(y[mask], same[mask]) and bool(torch.isnan(y[1, :, 1]).any())


def test_empty_and_leading_dimensions():
    g = torch.ones(8, device="cuda")
    x = torch.empty(0, 4, 8, device="cuda", dtype=F16)
    y, m, r = tg.group_norm_train(x, 2, g)
    assert y.shape == x.shape and m.shape == (0, 2)
    d = tg.group_norm_backward(x, x, 2, g, m, r)
    assert d.dx.shape == x.shape and not d.dgamma.any() and not d.dbeta.any()
    x = torch.randn(2, 3, 5, 8, device="cuda")
    assert torch.equal(tg.group_norm(x, 2, g).view(2, 15, 8), tg.group_norm(x.view(2, 15, 8), 2, g))
    one = x[:1, :1, :1].expand(1, 3, 5, 8)  # one row for all
    assert torch.equal(tg.group_norm(one, 2, g), tg.group_norm(one.contiguous(), 2, g))


def test_out():
    for case in (((2, 60, 16), 4, "f32", "silu", True, True, 0), ((9, 64), 4, "bf16", "none", True, True, 0)):
        c = Case(case)
        (x, G, ga), more = c.args(), c.more()
        want = tg.group_norm(x, G, ga, **more)
        a, z = x.clone(), more["z"].clone()
        assert torch.equal(tg.group_norm(a, G, ga, **more, out=a), want)
        assert torch.equal(tg.group_norm(x, G, ga, **dict(more, z=z), out=z), want)
        _, m, r = tg.group_norm_train(x, G, ga, **more)
        dy = up(c.dy)
        full = tg.group_norm_backward(dy, x, G, ga, m, r, **more)
        for t in (x, dy):
            xx, dd = x.clone(), dy.clone()
            got = tg.group_norm_backward(dd, xx, G, ga, m, r, **more, out=xx if t is x else dd)
            assert torch.equal(got.dx, full.dx) and torch.equal(got.dz, full.dz)
        with pytest.raises(ValueError, match="shares memory with x"):
            tg.group_norm_train(x, G, ga, **more, out=x)
        with pytest.raises(ValueError, match="shares memory with z"):
            tg.group_norm_backward(dy, x, G, ga, m, r, **more, out=more["z"])


def test_refusals():
    x, g = torch.zeros(2, 3, 8, device="cuda", dtype=F16), torch.ones(8, device="cuda")
    for f, text in ((lambda: tg.group_norm(x, 3, g), "must divide"), (lambda: tg.group_norm(x, 0, g), "must divide"),
                    (lambda: tg.group_norm(x[0, 0], 2, g), "x must be"), (lambda: tg.group_norm(x[:, :0], 2, g), "a row for each"),
                    (lambda: tg.group_norm(x, 2, None), "gamma is required"), (lambda: tg.group_norm(x, 2, g.half()), "gamma must be"),
                    (lambda: tg.group_norm(x, 2, g, z=x.float()), "z must be"), (lambda: tg.group_norm(x, 2, g, act="tanh"), "act must be"),
                    (lambda: tg.group_norm(x.transpose(0, 1), 2, g), "one stride apart"),
                    (lambda: tg.group_norm_backward(x, x, 2, g, g, g), "mean must have shape")):
        with pytest.raises(ValueError, match=text):
            f()


def test_captured_into_a_graph():
    """Replays with eager work between, on buffers that other calls use too."""
    cases = [Case(((2, 300, 32), 4, "bf16", "silu", True, True, 0)), Case(((40, 64), 4, "f16", "none", True, True, 0))]
    sets = [(c.args(), c.more(), up(c.dy)) for c in cases]

    def work():
        out = []
        for (x, G, ga), more, dy in sets:
            y, m, r = tg.group_norm_train(x, G, ga, **more)
            out += [y, m, r, *[t for t in tg.group_norm_backward(dy, x, G, ga, m, r, **more)]]
        return out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for k in range(3):
        for (x, _, _), _, _ in sets:
            x.copy_(torch.randn_like(x))
        want = [t.clone() for t in work()]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
