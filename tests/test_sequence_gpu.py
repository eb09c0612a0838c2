"""The sequence operators on the GPU against the 64-bit references of
seq_ref.py, with that file's bounds: every element, at sizes and masks where
they can go wrong (odd widths, one token, no token, strided slices, tails of
every tile, states, cache slots without a sequence)."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import seq_ref as R
from gpu_cases import note

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
TYPES = {"f16": F16, "bf16": BF16, "f32": F32}


class Rand:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, dtype=F32, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=self.g) * scale + shift).to(dtype)


def up(t, wide=0):
    """On the device; with ``wide``, as a slice of rows that are longer."""
    if t is None:
        return None
    t = t.cuda()
    if not wide:
        return t
    big = torch.full(t.shape[:-1] + (t.shape[-1] + wide,), float("nan"), dtype=t.dtype, device="cuda")
    big[..., wide:] = t
    return big[..., wide:]


def f64(t):
    return None if t is None else t.double()


# ---- layer norm

NORM = [
    # rows, C, type, residual, beta, extra row stride
    (1, 1, "f32", False, True, 0), (3, 2, "f16", True, True, 0), (5, 63, "bf16", False, False, 0),
    (4, 64, "f32", True, True, 0), (9, 65, "f16", True, True, 0), (7, 363, "f32", False, True, 0),
    (6, 512, "bf16", True, True, 8), (3, 514, "f16", False, True, 2), (2, 1000, "bf16", True, False, 0),
    (16, 1024, "f16", True, True, 0), (5, 2049, "bf16", False, True, 0), (3, 2052, "f32", True, True, 4),
    (3, 4096, "bf16", True, True, 0), (2, 8200, "f16", False, True, 0), (2, 9001, "f32", True, True, 0),
    (2, 20000, "bf16", True, True, 0), (1, 40000, "f32", False, True, 0), (2, 70001, "f16", True, True, 0),
    (2500, 48, "f16", True, True, 0), (1030, 1024, "bf16", True, True, 0),
]


def _norm_case(case):
    rows, C, dt, res, has_beta, wide = case
    r, dtype = Rand(rows * 31 + C), TYPES[dt]
    x = r(rows, C, dtype=dtype, shift=3.0)
    residual = r(rows, C, dtype=dtype, scale=2.0) if res else None
    gamma, beta = r(C, shift=1.0, scale=0.3), r(C) if has_beta else None
    s = x if residual is None else (x.float() + residual.float()).to(dtype)
    return r, dtype, x, residual, gamma, beta, s, wide


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(case):
    note("norm %s" % (case,))
    r, dtype, x, residual, gamma, beta, s, wide = _norm_case(case)
    dev = [up(x, wide), up(gamma), up(beta), 1e-5, up(residual, wide)]
    want = R.norm(s.double(), gamma.double(), f64(beta), 1e-5)
    y = tg.layer_norm(*dev)
    if residual is not None:
        y, total = y
        assert torch.equal(total.cpu(), s)
    R.check("y", y, *want["y"])
    y2, s2, mean, rstd = tg.layer_norm_train(*dev)
    assert torch.equal(y, y2) and torch.equal(s2.cpu(), s)
    R.check("mean", mean, *want["mean"])
    R.check("rstd", rstd, *want["rstd"])


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_backward(case):
    note("norm backward %s" % (case,))
    r, dtype, x, residual, gamma, beta, s, wide = _norm_case(case)
    dy = r(*x.shape, dtype=dtype)
    dsum = r(*x.shape, dtype=dtype) if residual is not None else None
    sd = up(s, wide)
    _, _, mean, rstd = tg.layer_norm_train(sd, up(gamma), up(beta))
    got = tg.layer_norm_backward(up(dy, wide), sd, up(gamma), mean, rstd, up(dsum, wide))
    want = R.norm_grads(dy.double(), s.double(), gamma.double(), 1e-5, f64(dsum))
    for name, g in zip(("dx", "dgamma", "dbeta"), got):
        R.check(name, g, *want[name])
    again = tg.layer_norm_backward(up(dy, wide), sd, up(gamma), mean, rstd, up(dsum, wide))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_norm_no_rows_and_leading_dimensions():
    g = torch.ones(8, device="cuda")
    x = torch.empty(0, 8, device="cuda", dtype=F16)
    y, s, mean, rstd = tg.layer_norm_train(x, g)
    assert y.shape == (0, 8) and mean.shape == (0,)
    dx, dg, db = tg.layer_norm_backward(x, x, g, mean, rstd)
    assert dx.shape == (0, 8) and not dg.any() and not db.any()
    x = Rand(1)(2, 3, 8).cuda()
    y, s, mean, rstd = tg.layer_norm_train(x, g)
    assert mean.shape == (2, 3)
    assert torch.equal(y.reshape(6, 8), tg.layer_norm(x.reshape(6, 8), g))
    one = x[:1, :1].expand(1, 5, 8)  # one row for all
    assert torch.equal(tg.layer_norm(one, g), y[:1, :1].expand(1, 5, 8))


def test_norm_large_mean():
    """A mean a thousand times the spread: the variance must not cancel."""
    x = Rand(3)(4, 2000, shift=1000.0)
    g = torch.ones(2000)
    want = R.norm(x.double(), g.double(), None, 1e-5)
    R.check("y", tg.layer_norm(up(x), up(g)), *want["y"])


# ---- short causal convolution

def _bounds(lengths):
    b = [0]
    for n in lengths:
        b.append(b[-1] + n)
    return b


CONV = [
    # lengths, packed, D, K, type, silu, bias, state, extra row stride
    ([1], False, 1, 2, "f32", True, True, False, 0), ([5, 5], False, 8, 4, "f16", True, True, True, 0),
    ([33], False, 64, 4, "bf16", True, False, False, 64), ([3, 3, 3], False, 37, 3, "f16", False, True, True, 0),
    ([2, 0, 1, 40, 3], True, 20, 4, "bf16", True, True, True, 0),
    ([0, 0, 7], True, 6, 8, "f32", True, True, True, 0), ([17, 64, 65, 130], True, 130, 4, "f16", True, True, False, 2),
    ([100], True, 1030, 5, "f32", True, True, False, 0), ([0], True, 4, 4, "f16", True, True, True, 0),
    ([300, 1, 211], True, 260, 6, "bf16", True, True, True, 4), ([64], False, 40, 7, "f16", True, True, False, 0),
    ([600, 600], False, 516, 2, "bf16", True, True, False, 0),
]


def _conv_case(case):
    lengths, packed, D, K, dt, act, has_bias, has_state, wide = case
    r, dtype = Rand(sum(lengths) * 7 + D), TYPES[dt]
    T, S = sum(lengths), len(lengths)
    x, w = r(T, D, dtype=dtype), r(K, D, scale=0.5)
    bias = r(D) if has_bias else None
    init = r(S, K - 1, D, dtype=dtype) if has_state else None
    b = _bounds(lengths)
    off = torch.tensor(b, dtype=torch.int32).cuda() if packed else None
    shape = (T, D) if packed else (S, T // S, D)
    parts = []
    for i in range(S):
        i0 = init[i].double() if has_state else torch.zeros(K - 1, D, dtype=F64)
        parts.append((b[i], b[i + 1], i0))
    return r, dtype, x, w, bias, init, off, shape, parts, act, wide


def _cat(pairs):
    return torch.cat([p[0] for p in pairs]), torch.cat([p[1] for p in pairs])


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(case):
    note("conv %s" % (case,))
    r, dtype, x, w, bias, init, off, shape, parts, act, wide = _conv_case(case)
    y, state = tg.causal_conv(up(x.reshape(shape), wide), up(w), up(bias), "silu" if act else "none",
                              up(init), off, return_state=True)
    want, last = [], []
    for lo, hi, i0 in parts:
        v, l, _ = R.conv(x[lo:hi].double(), w.double(), f64(bias), act, i0)
        want.append(v)
        last.append(l)
    R.check("y", y.reshape(x.shape), *_cat(want))
    assert torch.equal(state.cpu().double(), torch.stack(last))


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_backward(case):
    note("conv backward %s" % (case,))
    r, dtype, x, w, bias, init, off, shape, parts, act, wide = _conv_case(case)
    K, D = w.shape
    dy = r(*x.shape, dtype=dtype)
    dlast = r(len(parts), K - 1, D, dtype=dtype) if init is not None else None
    args = (up(dy.reshape(shape), wide), up(x.reshape(shape), wide), up(w), up(bias),
            "silu" if act else "none", up(init), off, up(dlast))
    dx, dw, dbias, dinit = tg.causal_conv_backward(*args)
    want = [R.conv_grads(dy[lo:hi].double(), x[lo:hi].double(), w.double(), f64(bias), act, i0,
                         None if dlast is None else dlast[i].double())
            for i, (lo, hi, i0) in enumerate(parts)]
    R.check("dx", dx.reshape(x.shape), *_cat([g["dx"] for g in want]))
    T = x.shape[0]
    for name, got in (("dw", dw), ("dbias", dbias)):
        v = sum(g[name][0] for g in want)
        mag = sum(g[name][0].abs() + g[name][1] / R.E for g in want)
        R.check(name, got, v, sum(g[name][1] for g in want) + 2 * len(want) * R.E * mag)
    if init is None:
        assert dinit is None
    else:
        R.check("dinit", dinit, torch.stack([g["dinit"][0] for g in want]),
                torch.stack([g["dinit"][1] for g in want]))
    again = tg.causal_conv_backward(*args)
    assert all(a is None or torch.equal(a, b) for a, b in zip((dx, dw, dbias, dinit), again))


@pytest.mark.parametrize("D,K,dt,act", [(1, 2, "f32", True), (64, 4, "bf16", True), (37, 4, "f16", False),
                                        (1028, 8, "f16", True), (130, 3, "bf16", True)])
def test_conv_step(D, K, dt, act):
    note("conv step D=%d K=%d %s" % (D, K, dt))
    r, dtype = Rand(D), TYPES[dt]
    n, num = 5, 9
    x, w, bias, state = r(n, D, dtype=dtype), r(K, D, scale=0.5), r(D), r(num, K - 1, D, dtype=dtype)
    slots = torch.tensor([3, -1, 0, 9, 8], dtype=torch.int32)
    st = up(state)
    y = tg.causal_conv_step(up(x, 4), st, up(w), up(bias), "silu" if act else "none", slots.cuda())
    want, bound, held = torch.zeros(n, D, dtype=F64), torch.zeros(n, D, dtype=F64), state.clone()
    for i, at in enumerate(slots.tolist()):
        if 0 <= at < num:
            (v, b), last, _ = R.conv(x[i:i + 1].double(), w.double(), bias.double(), act, state[at].double())
            want[i], bound[i], held[at] = v[0], b[0], last.to(dtype)
    R.check("y", y, want, bound)
    assert torch.equal(st.cpu(), held)
    st = up(state[:n])  # without slots: row i keeps state i
    y = tg.causal_conv_step(up(x), st, up(w), up(bias), "silu" if act else "none")
    (v, b), last, _ = R.conv(x[1:2].double(), w.double(), bias.double(), act, state[1].double())
    R.check("y", y[1:2], v, b)
    assert torch.equal(st[1].cpu(), last.to(dtype)) and y.shape == (n, D)
    assert tg.causal_conv_step(up(x[:0]), st, up(w), up(bias)).shape == (0, D)


# ---- selective scan

SCAN = [
    # lengths, packed, D, N, G, type, gate, softplus, state, extra row stride
    ([1], False, 1, 1, 1, "f32", True, True, False, 0), ([16], False, 16, 16, 1, "f32", False, True, False, 0),
    ([17, 17], False, 20, 16, 1, "f16", True, True, True, 0), ([50], False, 33, 5, 3, "bf16", True, True, True, 3),
    ([2, 0, 1, 40, 31], True, 34, 16, 2, "f16", True, True, True, 0), ([0, 5], True, 8, 4, 1, "f32", True, False, True, 0),
    ([0], True, 16, 16, 1, "bf16", True, True, True, 0), ([130], True, 48, 8, 1, "bf16", True, True, False, 8),
    ([33, 8], True, 18, 24, 1, "f32", True, True, True, 0), ([19], False, 16, 64, 1, "f32", True, True, True, 0),
    ([9, 12], True, 17, 128, 1, "f16", True, True, True, 0), ([23], False, 16, 100, 2, "f32", False, True, False, 0),
    ([600], False, 16, 16, 1, "f32", True, True, False, 0), ([257, 300], True, 80, 16, 1, "bf16", True, True, True, 0),
    ([70, 70, 70], False, 130, 2, 2, "f16", True, True, False, 0), ([1100, 3], True, 16, 4, 1, "f32", True, True, True, 0),
]


class ScanCase:
    def __init__(self, case):
        lengths, packed, D, N, G, dt, gate, soft, state, wide = case
        r, self.dtype = Rand(sum(lengths) * 5 + D + N), TYPES[dt]
        T, S = sum(lengths), len(lengths)
        self.T, self.S, self.D, self.N, self.G, self.r, self.soft = T, S, D, N, G, r, soft
        self.x, self.dt = r(T, D, dtype=self.dtype), r(T, D, dtype=self.dtype, scale=0.5)
        self.bias = r(D, shift=-3.0)
        if not soft:
            self.dt, self.bias = (self.dt.abs() * 0.1).to(self.dtype), self.bias.abs() * 0.01
        self.A = -torch.arange(1, N + 1).float().repeat(D, 1) * (1 + 0.1 * r(D, N).clamp(-2, 2))
        self.B, self.C = r(T, G, N, dtype=self.dtype), r(T, G, N, dtype=self.dtype)
        self.skip = r(D)
        self.z = r(T, D, dtype=self.dtype) if gate else None
        self.init = r(S, D, N) if state else None
        self.b = _bounds(lengths)
        self.off = torch.tensor(self.b, dtype=torch.int32).cuda() if packed else None
        self.lead = (T,) if packed else (S, T // S)
        self.wide = wide

    def dev(self, t):
        return None if t is None else up(t.reshape(self.lead + t.shape[1:]), self.wide)

    def bc(self, t):
        """B or C as a slice of a wider projection, groups together."""
        flat = t.reshape(self.lead + (self.G * self.N,))
        return up(flat, self.wide + 1).unflatten(-1, (self.G, self.N))

    def args(self):
        return (self.dev(self.x), self.dev(self.dt), up(self.A), self.bc(self.B), self.bc(self.C))

    def more(self):
        return dict(D=up(self.skip), z=self.dev(self.z), dt_bias=up(self.bias), softplus=self.soft,
                    initial_state=up(self.init), offsets=self.off)

    def ref(self, i, fn, *lead, **kw):
        lo, hi = self.b[i], self.b[i + 1]
        init = self.init[i].double() if self.init is not None else torch.zeros(self.D, self.N, dtype=F64)
        cut = lambda t: None if t is None else t[lo:hi].double()  # noqa: E731
        return fn(*(cut(t) for t in lead), cut(self.x), cut(self.dt), self.A.double(), cut(self.B),
                  cut(self.C), self.skip.double(), cut(self.z), self.bias.double(), self.soft, init, **kw)


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(case):
    note("scan %s" % (case,))
    c = ScanCase(case)
    y, state = tg.selective_scan(*c.args(), return_state=True, **c.more())
    refs = [c.ref(i, R.scan) for i in range(c.S)]
    R.check("y", y.reshape(c.x.shape), *_cat([r[0] for r in refs]))
    R.check("state", state, torch.stack([r[1][0] for r in refs]), torch.stack([r[1][1] for r in refs]))
    y2, s2, saved = tg.selective_scan_train(*c.args(), return_state=True, **c.more())
    assert torch.equal(y, y2) and torch.equal(state, s2)


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_backward(case):
    note("scan backward %s" % (case,))
    c = ScanCase(case)
    dy = c.r(*c.x.shape, dtype=c.dtype)
    dstate = c.r(c.S, c.D, c.N) if c.init is not None else None
    y, saved = tg.selective_scan_train(*c.args(), **c.more())
    got = tg.selective_scan_backward(c.dev(dy), *c.args(), saved, dstate=up(dstate), **c.more())
    refs = [c.ref(i, R.scan_grads, dy, dfinal=None if dstate is None else dstate[i].double())
            for i in range(c.S)]
    for name in ("dx", "ddt", "dz"):
        if getattr(got, name) is not None:
            R.check(name, getattr(got, name).reshape(c.x.shape), *_cat([r[name] for r in refs]))
    assert (got.dz is None) == (c.z is None)
    for name in ("dB", "dC"):
        R.check(name, getattr(got, name).reshape(c.T, c.G, c.N), *_cat([r[name] for r in refs]))
    for name, key in (("dA", "dA"), ("dD", "dD"), ("ddt_bias", "dbias")):
        v, e = sum(r[key][0] for r in refs), sum(r[key][1] for r in refs)
        R.check(name, getattr(got, name), v, e + (c.S + 1) * R.E * sum(r[key][0].abs() for r in refs))
    if c.init is not None:
        R.check("dinit", got.dinitial_state, torch.stack([r["dinit"][0] for r in refs]),
                torch.stack([r["dinit"][1] for r in refs]))
    again = tg.selective_scan_backward(c.dev(dy), *c.args(), saved, dstate=up(dstate), **c.more())
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("D,N,G,dt,gate", [(1, 1, 1, "f32", True), (64, 16, 1, "bf16", True), (70, 16, 2, "f16", False),
                                           (18, 5, 3, "f32", True), (130, 128, 1, "bf16", True), (16, 24, 1, "f16", True)])
def test_scan_step(D, N, G, dt, gate):
    note("scan step D=%d N=%d G=%d %s" % (D, N, G, dt))
    n, num = 5, 7
    c = ScanCase(([1] * n, True, D, N, G, dt, gate, True, False, 0))
    state = c.r(num, D, N)
    slots = [6, -1, 2, 7, 0]
    st = up(state)
    more = dict(D=up(c.skip), z=c.dev(c.z), dt_bias=up(c.bias))
    y = tg.selective_scan_step(*c.args(), st, slots=torch.tensor(slots, dtype=torch.int32).cuda(), **more)
    want, bound = torch.zeros(n, D, dtype=F64), torch.zeros(n, D, dtype=F64)
    held, eheld = state.double(), torch.zeros(num, D, N, dtype=F64)
    for i, at in enumerate(slots):
        if 0 <= at < num:
            c.init = torch.zeros(n, D, N)
            c.init[i] = state[at]
            (v, b), (h, eh), _ = c.ref(i, R.scan)
            want[i], bound[i], held[at], eheld[at] = v[0], b[0], h, eh
    R.check("y", y, want, bound)
    R.check("state", st, held, eheld)
    assert torch.equal(st[[1, 3, 4, 5]].cpu(), state[[1, 3, 4, 5]])


def test_scan_prompt_then_steps():
    """A prompt in two chunks and then single tokens give what one call gives."""
    c = ScanCase(([48, 48], False, 40, 16, 1, "f32", True, True, False, 0))
    x, dt, A, B, C = c.args()
    more = dict(D=up(c.skip), dt_bias=up(c.bias))
    z = c.dev(c.z)
    whole, last = tg.selective_scan(x, dt, A, B, C, z=z, return_state=True, **more)
    cut = lambda lo, hi: (x[:, lo:hi], dt[:, lo:hi], A, B[:, lo:hi], C[:, lo:hi])  # noqa: E731
    y0, state = tg.selective_scan(*cut(0, 21), z=z[:, :21], return_state=True, **more)
    y1, state = tg.selective_scan(*cut(21, 40), z=z[:, 21:40], initial_state=state, return_state=True, **more)
    ys = [y0, y1]
    for t in range(40, 48):
        ys.append(tg.selective_scan_step(x[:, t], dt[:, t], A, B[:, t], C[:, t], state, z=z[:, t], **more).unsqueeze(1))
    refs = [c.ref(i, R.scan) for i in range(2)]
    want, bound = _cat([r[0] for r in refs])
    R.check("y", torch.cat(ys, 1).reshape(96, 40), want, bound)
    R.check("state", state, torch.stack([r[1][0] for r in refs]), torch.stack([r[1][1] for r in refs]))
    R.check("whole", whole.reshape(96, 40), want, bound)


# ---- streams, graphs

def _everything(c, g, w, dy, dw_dy, conv_state, scan_state):
    """Every operator once, in a fixed order; the outputs."""
    args, more = c.args(), c.more()
    more.pop("initial_state")
    out = []
    y, s, mean, rstd = tg.layer_norm_train(args[0], g, residual=args[1])
    out += [y, s, *tg.layer_norm_backward(dy, s, g, mean, rstd)]
    out += list(tg.causal_conv(args[0], w, offsets=c.off, return_state=True))
    out += [t for t in tg.causal_conv_backward(dy, args[0], w, offsets=c.off) if t is not None]
    y, saved = tg.selective_scan_train(*args, **more)
    out += [y, *(t for t in tg.selective_scan_backward(dy, *args, saved, **more) if t is not None)]
    step = [t[:3] for t in (args[0], args[1])] + [args[2]] + [t[:3] for t in args[3:]]
    out.append(tg.causal_conv_step(step[0], conv_state, w))
    out.append(tg.selective_scan_step(*step, scan_state))
    return out


def _everything_case():
    c = ScanCase(([70, 0, 133], True, 48, 16, 1, "f16", True, True, True, 0))
    r = Rand(4)
    return (c, r(48).cuda(), r(4, 48).cuda(), r(203, 48, dtype=F16).cuda(), None,
            r(3, 3, 48, dtype=F16).cuda(), r(3, 48, 16).cuda())


def test_graph_replays_equal_eager():
    c = _everything_case()
    conv0, scan0 = c[5].clone(), c[6].clone()
    want = [t.clone() for t in _everything(*c)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    # The tensors that the case makes on its way to the device are made
    # outside the graph.
    args, more = c[0].args(), c[0].more()
    c[0].args, c[0].more = lambda: args, lambda: dict(more)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = _everything(*c)
    for i in range(3):
        c[5].copy_(conv0)
        c[6].copy_(scan0)
        for t in got:
            t.fill_(float("nan"))
        torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), "replay %d, output %d" % (i, k)


def test_other_stream():
    """Calls with a stream of their own, one after another without a wait in
    between on the host: results and scratch belong to that stream."""
    x = Rand(9)(3000, 1000, dtype=BF16).cuda()
    g = torch.ones(1000, device="cuda")
    y, s, mean, rstd = tg.layer_norm_train(x, g)
    want = tg.layer_norm_backward(x, s, g, mean, rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [tg.layer_norm_backward(x, s, g, mean, rstd, stream=side) for _ in range(4)]
    junk = [torch.full((4, 1000, 1000), float("nan"), device="cuda") for _ in range(4)]
    side.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    del junk


def test_refuses_host_and_mismatched_tensors():
    x = torch.zeros(2, 4, 8, device="cuda", dtype=F16)
    w = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="w must be on"):
        tg.causal_conv(x, w.cpu())
    with pytest.raises(ValueError, match="w must be torch.float32"):
        tg.causal_conv(x, w.half())
    with pytest.raises(ValueError, match="last dimension"):
        tg.causal_conv(x.transpose(1, 2), torch.zeros(4, 4, device="cuda"))
    with pytest.raises(ValueError, match="with offsets"):
        tg.causal_conv(x[0], w)
    with pytest.raises(ValueError, match="offsets must be"):
        tg.causal_conv(x[0], w, offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="initial_state must have shape"):
        tg.causal_conv(x, w, initial_state=torch.zeros(2, 4, 8, device="cuda", dtype=F16))
    with pytest.raises(ValueError, match="act must be"):
        tg.causal_conv(x, w, act="relu")
    with pytest.raises(tg.TgError, match="TG_ERR_UNSUPPORTED"):
        tg.causal_conv(x, torch.zeros(9, 8, device="cuda"))
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        tg.layer_norm(x.double(), w[0])
    with pytest.raises(ValueError, match="one stride apart"):
        tg.layer_norm(torch.zeros(4, 4, 8, device="cuda", dtype=F16)[:, :2], w[0])
    b = torch.zeros(2, 4, 1, 4, device="cuda", dtype=F16)
    a = torch.zeros(8, 4, device="cuda")
    with pytest.raises(ValueError, match="dt must have shape"):
        tg.selective_scan(x, x[:, :3], a, b, b)
    with pytest.raises(ValueError, match="groups of B"):
        tg.selective_scan(x, x, a, torch.zeros(2, 4, 3, 4, device="cuda", dtype=F16), b)
    with pytest.raises(tg.TgError, match="TG_ERR_UNSUPPORTED"):
        big = torch.zeros(2, 4, 1, 129, device="cuda", dtype=F16)
        tg.selective_scan(x, x, torch.zeros(8, 129, device="cuda"), big, big)
    with pytest.raises(tg.TgError, match="TG_ERR_INVALID_ARGUMENT"):  # fewer slots than rows
        tg.selective_scan_step(x[0], x[0], a, b[0], b[0], torch.zeros(2, 8, 4, device="cuda"))
    with pytest.raises(ValueError, match="saved must have shape"):
        tg.selective_scan_backward(x, x, x, a, b, b, torch.zeros(5, device="cuda"))


# ---- many sequences, far rows, wrong offsets

def _many(S, L, D, N, dt=F32, seed=5):
    r = Rand(seed)
    dev = lambda *s, **k: r(*s, **k).cuda()  # noqa: E731
    x = [dev(S, L, D, dtype=dt), dev(S, L, D, dtype=dt, scale=0.5),
         -torch.arange(1, N + 1).float().repeat(D, 1).cuda(), dev(S, L, 1, N, dtype=dt), dev(S, L, 1, N, dtype=dt)]
    return x, dict(D=dev(D), z=dev(S, L, D, dtype=dt), dt_bias=dev(D, shift=-3.0), initial_state=dev(S, D, N)), dev(S, L, D, dtype=dt)


@pytest.mark.parametrize("N", [3, 8, 16, 30, 64, 128])
def test_scan_many_sequences(N):
    """So many sequences that single waves take them whole: against the 64-bit
    reference for some, and dA, dD and ddt_bias against the sum over small batches."""
    S, L, D = 4100, 19, 16
    note("scan of %d sequences, N=%d" % (S, N))
    args, more, dy = _many(S, L, D, N)
    y, state, saved = tg.selective_scan_train(*args, return_state=True, **more)
    g = tg.selective_scan_backward(dy, *args, saved, **more)
    for i in (0, 1, 2047, S - 1):
        cut = lambda t: t[i].double().cpu()  # noqa: E731
        ref = (cut(args[0]), cut(args[1]), args[2].double().cpu(), cut(args[3]), cut(args[4]), more["D"].double().cpu(),
               cut(more["z"]), more["dt_bias"].double().cpu(), True, cut(more["initial_state"]))
        (v, b), (h, eh), _ = R.scan(*ref)
        R.check("y", y[i], v, b)
        R.check("state", state[i], h, eh)
        w = R.scan_grads(cut(dy), *ref)
        for name, got in (("dx", g.dx), ("ddt", g.ddt), ("dz", g.dz), ("dB", g.dB), ("dC", g.dC), ("dinit", g.dinitial_state)):
            R.check(name, got[i], *w[name])
    total = None
    for lo in range(0, S, 205):
        hi = min(S, lo + 205)
        part = [t[lo:hi] if t.dim() > 2 else t for t in args]
        m = {k: t[lo:hi] if t.dim() > 1 else t for k, t in more.items()}
        _, sv = tg.selective_scan_train(*part, **m)
        p = tg.selective_scan_backward(dy[lo:hi], *part, sv, **m)
        three = [p.dA.double(), p.dD.double(), p.ddt_bias.double()]
        total = three if total is None else [a + b for a, b in zip(total, three)]
    for name, got, want in zip(("dA", "dD", "ddt_bias"), (g.dA, g.dD, g.ddt_bias), total):
        # 4100 * 19 terms of either sign, each side's sums in fp32 trees of under 2^11 terms a level.
        assert float((got.double() - want).norm()) <= 1e-5 * float(want.norm()) + 1e-6, name


def test_rows_far_apart():
    """Row strides that put the last rows past 2^31 elements and 2^32 bytes."""
    rows, stride, D = 1500, 1500000, 24
    big = torch.empty(rows, stride, dtype=F16, device="cuda")
    r = Rand(8)
    small = [r(rows, D, dtype=F16) for _ in range(3)]
    view = []
    for k, t in enumerate(small):
        view.append(big[:, 1000 * k:1000 * k + D])
        view[k].copy_(t)
    near = [t.cuda() for t in small]
    off = torch.tensor([0, 700, 700, 701, rows], dtype=torch.int32, device="cuda")
    w, g = r(4, D).cuda(), r(D).cuda()
    same = lambda f: [(a, b) for a, b in zip(f(near), f(view))]  # noqa: E731
    A = -torch.ones(D, 4).cuda()
    bc = lambda t: t[:, :4].unflatten(-1, (1, 4))  # noqa: E731

    def everything(v):
        y, s, mean, rstd = tg.layer_norm_train(v[0], g, residual=v[1])
        out = [y, s, *tg.layer_norm_backward(v[2], v[0], g, mean, rstd, dsum=v[1])]
        out += [tg.causal_conv(v[0], w, offsets=off), *tg.causal_conv_backward(v[1], v[0], w, offsets=off)[:3]]
        sy, saved = tg.selective_scan_train(v[0], v[1], A, bc(v[1]), bc(v[2]), z=v[2], offsets=off)
        d = tg.selective_scan_backward(v[1], v[0], v[1], A, bc(v[1]), bc(v[2]), saved, z=v[2], offsets=off)
        return out + [sy, d.dx, d.ddt, d.dA, d.dB, d.dC, d.dz]
    for k, (a, b) in enumerate(same(everything)):
        assert torch.equal(a, b), k
    with pytest.raises(tg.TgError, match="TG_ERR_UNSUPPORTED"):  # rows too far apart for the scan
        far = torch.empty(2, 1 << 25, dtype=F16, device="cuda")[:, :D]
        tg.selective_scan(far, far, A, bc(far), bc(far), offsets=off[:2])


@pytest.mark.parametrize("wrong", [[5, 9, 40], [0, 50, 20], [-7, 3, 1000], [30, 10, 0], [40, 40, 40]], ids=str)
def test_wrong_offsets_stay_inside(wrong):
    """Offsets that break the contract are cut to the rows: results are not
    specified, but nothing past the outputs is written."""
    note("wrong offsets %s" % wrong)
    rows, D, N = 40, 16, 16
    c = ScanCase(([rows], True, D, N, 1, "f32", True, True, False, 0))
    off = torch.tensor(wrong, dtype=torch.int32, device="cuda")
    guard = torch.full((3 * rows, D), 7.0, device="cuda")
    out = guard[rows:2 * rows]
    args, more = c.args(), c.more()
    more.pop("initial_state"), more.pop("offsets")
    tg.selective_scan(*args, offsets=off, out=out, **more)
    y, saved = tg.selective_scan_train(*args, offsets=off, **more)
    tg.selective_scan_backward(c.dev(c.x), *args, saved, offsets=off, **more)
    tg.causal_conv(args[0], torch.ones(4, D, device="cuda"), offsets=off, out=out, return_state=True)
    tg.causal_conv_backward(args[1], args[0], torch.ones(4, D, device="cuda"), offsets=off)
    torch.cuda.synchronize()
    assert bool((guard[:rows] == 7).all()) and bool((guard[2 * rows:] == 7).all())
