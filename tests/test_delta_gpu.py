"""The gated delta rule on the GPU against the 64-bit reference of delta_ref.py with
that file's tolerances, at sizes and inputs where it can go wrong: odd widths, one
token, no token, tails of a chunk, shared key heads, strided slices, states, cache
slots without a sequence, decays at both ends."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import delta_ref as D
from gpu_cases import note

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
TYPES = {"f16": F16, "bf16": BF16, "f32": F32}


def up(t, wide=0):
    """On the device; with ``wide``, as a slice of rows that are longer, among NaN."""
    if t is None:
        return None
    t = t.cuda()
    if not wide:
        return t
    lead = t.dim() - (2 if t.dim() > 2 else 1)
    flat = t.reshape(t.shape[:lead] + (-1,))
    big = torch.full(flat.shape[:-1] + (flat.shape[-1] + wide,), float("nan"), dtype=t.dtype, device="cuda")
    big[..., wide:] = flat
    return big[..., wide:].unflatten(-1, t.shape[lead:])


class Case:
    """lengths, packed, key heads, value heads, K, V, type, state, plain gates and
    keys, extra row width."""

    def __init__(self, case, seed=0):
        lengths, self.packed, HK, HV, K, V, dt, state, self.plain, wide = case
        self.T, self.dtype, self.lengths, self.HV = sum(lengths), TYPES[dt], lengths, HV
        self.bounds = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        g = torch.Generator().manual_seed(seed + self.T * 31 + K * 7 + V)
        r = lambda *s, scale=1.0, shift=0.0: (torch.randn(*s, generator=g) * scale + shift)  # noqa: E731
        T, S, t = self.T, len(lengths), self.dtype
        # Plain keys are of length 1 at the most, or the map of the state would grow it.
        self.q = r(T, HK, K).to(t)
        k = r(T, HK, K)
        self.k = (k / (k.norm(dim=-1, keepdim=True) + 1e-3) if self.plain else k).to(t)
        self.v = r(T, HV, V).to(t)
        self.dt = (torch.rand(T, HV, generator=g) * 0.4 if self.plain else r(T, HV, scale=0.5)).to(t)
        self.beta = (torch.rand(T, HV, generator=g) if self.plain else r(T, HV)).to(t)
        self.A = -torch.rand(HV, generator=g) * 8
        self.dt_bias = None if self.plain else r(HV, shift=-2.0)
        self.initial = r(S, HV, K, V, scale=0.3) if state else None
        self.dy = r(T, HV, V).to(t)
        self.dstate = r(S, HV, K, V, scale=0.3) if state else None
        self.wide = wide
        self.offsets = torch.tensor(self.bounds, dtype=torch.int32, device="cuda") if self.packed else None

    def dev(self, t, wide=None):
        if not self.packed:
            t = t.reshape((len(self.lengths), -1) + t.shape[1:])
        return up(t, self.wide if wide is None else wide)

    def args(self):
        return (self.dev(self.q), self.dev(self.k), self.dev(self.v), self.dev(self.dt), up(self.A), self.dev(self.beta))

    def more(self):
        m = dict(dt_bias=up(self.dt_bias), initial_state=up(self.initial), offsets=self.offsets)
        if self.plain:
            m.update(softplus=False, sigmoid=False, normalize=False, scale=0.7)
        return m

    def want(self, gradient=False):
        leaf = lambda t: None if t is None else t.double().requires_grad_(gradient)  # noqa: E731
        x = [leaf(t) for t in (self.q, self.k, self.v, self.dt, self.A, self.beta)]
        bias, initial = leaf(self.dt_bias), leaf(self.initial)
        flags = dict(softplus=False, sigmoid=False, normalize=False, scale=0.7) if self.plain else {}
        y, state, g, kap, chunks = D.delta(self.bounds, *x, dt_bias=bias, initial=initial, **flags)
        return x, bias, initial, y, state, g, kap, chunks


CASES = [
    ([1], False, 1, 1, 1, 1, "f32", False, False, 0), ([5, 5], False, 1, 2, 8, 16, "f16", True, False, 0),
    ([64], False, 2, 2, 64, 64, "bf16", True, False, 0), ([65, 65], False, 1, 1, 64, 32, "f32", False, False, 0),
    ([3, 0, 130, 1, 31], True, 2, 4, 20, 13, "f32", True, False, 0), ([3, 0, 130, 1, 31], True, 2, 4, 20, 13, "bf16", True, True, 3),
    ([0, 0, 7], True, 3, 3, 33, 50, "f16", True, False, 5), ([129], False, 2, 2, 128, 128, "bf16", False, False, 16),
    ([97], False, 1, 3, 128, 40, "f16", True, True, 8), ([70, 70], False, 1, 1, 128, 31, "f32", True, False, 0),
    ([40, 2], True, 1, 2, 200, 33, "bf16", True, False, 0), ([33, 64], True, 1, 1, 256, 48, "f16", False, False, 0),
    ([50], False, 1, 2, 130, 20, "f32", True, True, 1), ([96, 32], True, 2, 2, 256, 17, "f32", True, False, 8),
    ([66], False, 1, 4, 96, 256, "bf16", True, False, 0), ([0], True, 1, 2, 8, 16, "f16", True, False, 0),
    ([300], False, 1, 1, 16, 16, "f32", True, False, 0), ([17], True, 4, 4, 63, 65, "f32", False, True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    note("delta %s" % (case,))
    c = Case(case)
    _, _, _, y, state, _, kap, chunks = c.want()
    got, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
    shape = c.dev(c.v, 0).shape
    D.near("y", got, y.reshape(shape), D.allowed(c.dtype, kap, chunks, only="y", prompt=True), c.dtype)
    D.near("state", s, state, D.allowed(c.dtype, kap, chunks, prompt=True), F32)
    t, s2, saved = tg.gated_delta_rule_train(*c.args(), return_state=True, **c.more())
    D.near("y", t, y.reshape(shape), D.allowed(c.dtype, kap, chunks, only="y"), c.dtype)
    D.near("state", s2, state, D.allowed(c.dtype, kap, chunks), F32)
    again, s3 = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
    assert torch.equal(got, again) and torch.equal(s, s3)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    note("delta backward %s" % (case,))
    c = Case(case)
    x, bias, initial, y, state, g, kap, chunks = c.want(True)
    leaves = x + [t for t in (bias, initial) if t is not None]
    total = (y * c.dy.double()).sum() + (0 if c.dstate is None else (state * c.dstate.double()).sum())
    if c.T:
        want = torch.autograd.grad(total, leaves + list(g), allow_unused=True)
        dg, units = want[len(leaves)], want[len(leaves) + 1:]
    else:
        want = [torch.zeros_like(t) for t in x] + [torch.zeros_like(t) for t in leaves[6:-1]] + [c.dstate.double()]
        units = [torch.zeros_like(t) for t in x[:2]]
    _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
    more = c.more()
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **more)
    rel = D.allowed(c.dtype, kap, chunks, gradient=True)
    part = D.allowed(c.dtype, kap, chunks, gradient=True, only="qk")
    shaped = lambda w, t: w.reshape(c.dev(t, 0).shape)  # noqa: E731
    for name, at, t, u in (("dq", 0, c.q, units[0]), ("dk", 1, c.k, units[1])):
        size = None if c.plain else shaped(D.unit_size(x[at].detach(), u), t)
        D.near(name, getattr(got, name), shaped(want[at], t), part, c.dtype, size=size)
    D.near("dv", got.dv, shaped(want[2], c.v), rel, c.dtype)
    D.near("ddt", got.ddt, shaped(want[3], c.dt), rel, c.dtype)
    D.near("dbeta", got.dbeta, shaped(want[5], c.beta), rel, c.dtype)
    if c.T:
        raw = c.dt.double() if c.dt_bias is None else c.dt.double() + c.dt_bias.double()
        d = raw if c.plain else torch.nn.functional.softplus(raw, threshold=1e9)
        D.near("dA", got.dA, want[4], rel, F32, size=(dg * d).abs().sum(0).detach())
        if bias is not None:
            D.near("ddt_bias", got.ddt_bias, want[6], rel, F32, size=want[3].abs().sum(0))
    else:
        assert not got.dA.any()
    if initial is None:
        assert got.dinitial_state is None
    else:
        D.near("dinitial", got.dinitial_state, want[6 + (bias is not None)], rel, F32)
    again = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **more)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


# Few long sequences, which are walked in segments.
LONG = [
    ([1500], False, 1, 1, 32, 16, "f32", True, False, 0), ([1000, 30, 0, 500], True, 1, 2, 64, 40, "bf16", True, False, 3),
    ([1100], False, 1, 2, 100, 33, "f16", False, False, 0), ([700, 700], False, 1, 1, 130, 20, "bf16", True, True, 0),
    ([1300], False, 1, 1, 256, 17, "f32", True, False, 0), ([1, 1400, 1], True, 1, 1, 16, 70, "f16", True, False, 0),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_forward(case):
    test_forward(case)


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_backward(case):
    test_backward(case)


def test_long_wrong_offsets_stay_inside():
    c = Case(([2000], True, 1, 1, 16, 16, "f32", False, False, 0))
    guard = torch.full((6000, 1, 16), 7.0, device="cuda")
    for wrong in ([5, 900, 4000], [0, 1990, 20], [-7, 3, 9000], [1700, 10, 0]):
        off = torch.tensor(wrong, dtype=torch.int32, device="cuda")
        more = dict(c.more(), offsets=off)
        tg.gated_delta_rule(*c.args(), out=guard[2000:4000], **more)
        _, saved = tg.gated_delta_rule_train(*c.args(), **more)
        tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, **more)
    torch.cuda.synchronize()
    assert bool((guard[:2000] == 7).all()) and bool((guard[4000:] == 7).all())


STEPS = [(1, 1, 1, 1, 1, "f32", 0), (3, 2, 4, 20, 13, "bf16", 5), (5, 2, 2, 64, 64, "f16", 0), (2, 1, 2, 128, 128, "bf16", 16),
         (4, 1, 1, 256, 40, "f32", 4), (3, 1, 3, 130, 33, "f16", 0), (2, 4, 8, 96, 132, "f32", 0), (9, 1, 1, 8, 260, "bf16", 0)]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_step(case):
    n, HK, HV, K, V, dt, wide = case
    note("delta step %s" % (case,))
    c = Case(([1] * n, True, HK, HV, K, V, dt, True, False, wide))
    cache = torch.randn(n + 2, HV, K, V, generator=torch.Generator().manual_seed(n))
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32)
    slots[0] = -1 if n % 2 else n + 2  # no sequence here
    c.initial = cache[slots.long().clamp(0, n + 1)]
    _, _, _, y, state, _, kap, _ = c.want()
    dev, more = cache.cuda(), c.more()
    more.pop("initial_state"), more.pop("offsets")
    got = tg.gated_delta_rule_step(*c.args(), dev, slots=slots.cuda(), **more)
    assert not got[0].any()
    rel = D.allowed(F32, 1.0, 1)
    D.near("y", got[1:], y[1:], rel, c.dtype)
    after = cache.double()
    after[slots[1:].long()] = state[1:]
    D.near("state", dev, after, rel, F32)
    untouched = [i for i in range(n + 2) if i not in slots[1:].tolist()]
    assert torch.equal(dev[untouched].cpu(), cache[untouched])


def test_pieces_and_steps():
    """A prompt whole, in pieces that end inside a chunk, and token by token."""
    c = Case(([150, 150], False, 2, 4, 40, 24, "f32", True, False, 0))
    more = c.more()
    init = more.pop("initial_state")
    whole, last = tg.gated_delta_rule(*c.args(), return_state=True, initial_state=init, **more)
    cut = lambda lo, hi: [t if t.dim() == 1 else t[:, lo:hi] for t in c.args()]  # noqa: E731
    state, ys = init, []
    for lo, hi in ((0, 1), (1, 71), (71, 135)):
        y, state = tg.gated_delta_rule(*cut(lo, hi), return_state=True, initial_state=state, **more)
        ys.append(y)
    cache = torch.zeros(4, 4, 40, 24, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    cache[slots.long()] = state
    more.pop("offsets")
    for t in range(135, 150):
        tok = [u if u.dim() == 1 else u[:, t] for u in c.args()]
        ys.append(tg.gated_delta_rule_step(*tok, cache, slots=slots, **more).unsqueeze(1))
    rel = D.allowed(F32, 4.0, 6)
    D.near("y", torch.cat(ys, 1), whole.double().cpu(), rel, F32)
    D.near("state", cache[slots.long()], last.double().cpu(), rel, F32)


def test_packed_equals_dense():
    for dt in ("bf16", "f16", "f32"):
        c = Case(([70, 70, 70], False, 1, 2, 64, 32, dt, True, False, 0))
        off = torch.arange(0, 211, 70, dtype=torch.int32, device="cuda")
        flat = lambda t: t if t.dim() == 1 else t.flatten(0, 1)  # noqa: E731
        a, b = [t for t in c.args()], [flat(t) for t in c.args()]
        more, packed = c.more(), dict(c.more(), offsets=off)
        ya, sa, ka = tg.gated_delta_rule_train(*a, return_state=True, **more)
        yb, sb, kb = tg.gated_delta_rule_train(*b, return_state=True, **packed)
        assert torch.equal(ya.flatten(0, 1), yb) and torch.equal(sa, sb)
        ga = tg.gated_delta_rule_backward(c.dev(c.dy), *a, ka, **more)
        gb = tg.gated_delta_rule_backward(flat(c.dev(c.dy)), *b, kb, **packed)
        for name in ("dq", "dk", "dv", "ddt", "dbeta"):
            assert torch.equal(getattr(ga, name).flatten(0, 1), getattr(gb, name)), name
        assert torch.equal(ga.dinitial_state, gb.dinitial_state)


def test_no_decay_identical_keys_and_zero_keys():
    """The worst condition: one key for all tokens, b near 1, no decay; then zeros."""
    for dt in ("bf16", "f32"):
        c = Case(([140], False, 1, 1, 32, 16, dt, True, False, 0))
        c.k = c.k[:1].expand_as(c.k).contiguous()
        c.beta = torch.full_like(c.beta, 6.0)
        c.A = torch.zeros(1)
        _, _, _, y, state, _, kap, chunks = c.want()
        got, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
        D.near("y", got, y.reshape(got.shape), D.allowed(c.dtype, kap, chunks, only="y", prompt=True), c.dtype)
        D.near("state", s, state, D.allowed(c.dtype, kap, chunks, prompt=True), F32)
        c.k = torch.zeros_like(c.k)
        _, _, _, y, state, _, _, _ = c.want()
        got, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
        D.near("y", got, y.reshape(got.shape), D.allowed(c.dtype, 1.0, chunks, only="y", prompt=True), c.dtype)
        D.near("state", s, state, D.allowed(c.dtype, 1.0, chunks, prompt=True), F32)


def test_decays_at_both_ends():
    """Rates of -inf forget the state before every token, a step of zero keeps it,
    and strong decays leave the small ones after them exact."""
    c = Case(([100], False, 1, 3, 16, 8, "f32", True, False, 0))
    c.plain = True
    c.k, c.q = c.k * 0.2, c.q * 0.2
    c.dt_bias = None
    c.A = torch.tensor([-float("inf"), -1.0, -1e5])
    step = torch.rand(100, 3, generator=torch.Generator().manual_seed(2)) * 0.01
    step[::7] = 0.0
    step[5::11] += 5.0
    c.dt, c.beta = step, torch.rand(100, 3, generator=torch.Generator().manual_seed(3))
    _, _, _, y, state, _, kap, chunks = c.want()
    got, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
    rel = D.allowed(F32, kap, chunks)
    D.near("y", got, y.reshape(got.shape), rel, F32)
    D.near("state", s, state, rel, F32)
    cache = up(c.initial).clone()
    tok = [t if t.dim() == 1 else t[:, 0] for t in c.args()]
    flags = dict(softplus=False, sigmoid=False, normalize=False, scale=0.7)
    first = tg.gated_delta_rule_step(*tok, cache, **flags)
    D.near("y", first, y[:1], rel, F32)


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("lengths", [[1100], [4096], [65, 300]], ids=str)
def test_growing_decays(lengths, train):
    """Decays above 1, over chunks and over segments. An error of a share u of the
    largest state grows by no more than all decays together, e^G, up to the end: the
    state may be off by e^G times what it may be off without growth, of the largest
    state; y, q of length 1 and scale 1, by as much in every row."""
    c = Case((lengths, True, 2, 2, 16, 24, "f32", True, False, 0))
    rate = 3.0 / max(max(lengths), 1000)
    c.dt_bias, c.A = None, torch.tensor([1.0, 0.5])
    c.dt = torch.full((c.T, 2), rate)
    more = dict(initial_state=up(c.initial), offsets=c.offsets, softplus=False, scale=1.0)
    if train:
        got, s, _ = tg.gated_delta_rule_train(*c.args(), return_state=True, **more)
    else:
        got, s = tg.gated_delta_rule(*c.args(), return_state=True, **more)
    q, k, v, dt, A, beta, initial = (t.double() for t in (c.q, c.k, c.v, c.dt, c.A, c.beta, c.initial))
    args = (q, k, v, dt, A, beta, None, False, True, True, 1.0, initial)
    y, state, _, kap, chunks = D.delta(c.bounds, *args)
    # The largest state of each sequence, from the chunks' ends: between them it grows
    # by less than e^(32 rate) < 1.4 and what the values add.
    for i, (lo, hi) in enumerate(zip(c.bounds[:-1], c.bounds[1:])):
        _, g, b = D.gates(dt[lo:hi], A, beta[lo:hi], None, False, True)
        S, most = initial[i], initial[i].norm()
        for at in range(lo, hi, 32):
            to = min(at + 32, hi)
            S = D.walk(D.unit(q[at:to], True), D.unit(k[at:to], True), v[at:to], g[at - lo:to - lo],
                       b[at - lo:to - lo], 1.0, S)[1]
            most = torch.maximum(most, S.norm() + v[at:to].norm())
        bound = float(1.4 * most * torch.exp(g.sum(0)).max()) * D.allowed(F32, kap, chunks)
        off = (s[i].double().cpu() - state[i]).norm()
        assert off <= bound + D.E * state[i].norm(), (float(off), bound)
        rows = (got[lo:hi].double().cpu() - y[lo:hi]).flatten(1).norm(dim=1)
        assert bool((rows <= bound + D.E * y[lo:hi].flatten(1).norm(dim=1)).all()), (float(rows.max()), bound)


def test_a_bad_value_stays_in_its_sequence_and_head():
    c = Case(([70, 70, 70], True, 2, 2, 32, 16, "bf16", False, False, 0))
    off = torch.tensor(c.bounds, dtype=torch.int32, device="cuda")
    clean = tg.gated_delta_rule(*c.args(), **dict(c.more(), offsets=off))
    for bad in (float("nan"), float("inf")):
        args = list(c.args())
        args[2] = args[2].clone()
        args[2][75, 1, 3] = bad
        y = tg.gated_delta_rule(*args, **dict(c.more(), offsets=off))
        assert torch.equal(y[:70], clean[:70]) and torch.equal(y[140:], clean[140:])
        assert torch.equal(y[:, 0], clean[:, 0])
        assert not torch.isfinite(y[75:140, 1, 3]).all()


def test_rows_that_no_sequence_covers_are_left():
    c = Case(([20, 30], True, 1, 2, 16, 20, "f16", False, False, 0))
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    out = torch.full((50, 2, 20), 7.0, dtype=F16, device="cuda")
    tg.gated_delta_rule(*c.args(), **dict(c.more(), offsets=off, out=out))
    assert bool((out[40:] == 7).all()) and not bool((out[:40] == 7).all())


@pytest.mark.parametrize("wrong", [[5, 9, 40], [0, 50, 20], [-7, 3, 1000], [30, 10, 0], [40, 40, 40]], ids=str)
def test_wrong_offsets_stay_inside(wrong):
    note("wrong offsets %s" % wrong)
    c = Case(([40], True, 1, 2, 16, 20, "bf16", False, False, 0))
    off = torch.tensor(wrong, dtype=torch.int32, device="cuda")
    guard = torch.full((120, 2, 20), 7.0, dtype=BF16, device="cuda")
    more = dict(c.more(), offsets=off)
    more.pop("initial_state")
    tg.gated_delta_rule(*c.args(), out=guard[40:80], **more)
    _, saved = tg.gated_delta_rule_train(*c.args(), **more)
    tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, **more)
    torch.cuda.synchronize()
    assert bool((guard[:40] == 7).all()) and bool((guard[80:] == 7).all())


def test_out():
    c = Case(([80, 80], False, 1, 2, 32, 40, "bf16", False, False, 8))
    want = tg.gated_delta_rule(*c.args(), **c.more())
    args = c.args()
    assert tg.gated_delta_rule(*args, out=args[2], **c.more()) is args[2] and torch.equal(args[2], want)
    q, k, v, dt, A, beta = args = c.args()
    base = torch.zeros(2, 80, 200, dtype=BF16, device="cuda")
    cut = lambda lo: base[..., lo:lo + 80].unflatten(-1, (2, 40))  # noqa: E731
    with pytest.raises(ValueError, match="shares memory with q"):
        tg.gated_delta_rule(base[..., :32].unflatten(-1, (1, 32)), k, v, dt, A, beta, **c.more(), out=cut(20))
    with pytest.raises(ValueError, match="shares memory with v"):  # training reads v again
        tg.gated_delta_rule_train(*args, out=v, **c.more())
    with pytest.raises(ValueError, match="shares memory with v"):
        tg.gated_delta_rule(q, k, cut(1), dt, A, beta, **c.more(), out=cut(0))
    with pytest.raises(ValueError, match="shares memory with v"):
        tok = [t if t.dim() == 1 else t[:, 0] for t in args]
        tg.gated_delta_rule_step(*tok, torch.zeros(2, 2, 32, 40, device="cuda"), dt_bias=up(c.dt_bias), out=tok[2])


def test_refusals():
    c = Case(([6], False, 1, 2, 8, 4, "f16", True, False, 0))
    q, k, v, dt, A, beta = c.args()
    f = lambda **kw: tg.gated_delta_rule(**dict(dict(q=q, k=k, v=v, dt=dt, A=A, beta=beta), **kw))  # noqa: E731
    for bad, text in ((dict(q=q.float()), "q must be"), (dict(k=k[..., :4]), "q must have shape"), (dict(A=A.half()), "A must be"),
                      (dict(beta=beta[..., :1]), "beta must have shape"), (dict(v=v[:, :, 0]), "v must be"),
                      (dict(initial_state=torch.zeros(1, 2, 4, 8, device="cuda")), "initial_state must have shape"),
                      (dict(dt_bias=torch.zeros(3, device="cuda")), "dt_bias must have shape"), (dict(dt=None), "dt is required"),
                      (dict(k=k.expand(1, 6, 3, 8).contiguous(), q=q.expand(1, 6, 3, 8).contiguous()), "must divide"),
                      (dict(v=v.transpose(-1, -2).contiguous().transpose(-1, -2)), "heads of a row|contiguous"),
                      (dict(offsets=torch.zeros(2, device="cuda")), "v must be")):
        with pytest.raises(ValueError, match=text):
            f(**bad)
    with pytest.raises(tg.TgError, match="TG_ERR_UNSUPPORTED"):
        big = torch.zeros(1, 2, 1, 300, dtype=F16, device="cuda")
        tg.gated_delta_rule(big, big, big, dt[:, :2, :1], A[:1], beta[:, :2, :1])
    _, saved = tg.gated_delta_rule_train(q, k, v, dt, A, beta)
    with pytest.raises(ValueError, match="saved must have shape"):
        tg.gated_delta_rule_backward(v, q, k, v, dt, A, beta, saved[:-1])


def test_captured_into_a_graph():
    """Replayed with other work between, every replay against the eager result; two
    graphs on one pool."""
    c = Case(([100, 37], True, 1, 2, 64, 32, "bf16", True, False, 0))
    args, more, dy = c.args(), c.more(), c.dev(c.dy)
    cache = up(c.initial).clone()
    tok = [t if t.dim() == 1 else t[:2] for t in args]

    def work():
        y, s, saved = tg.gated_delta_rule_train(*args, return_state=True, **more)
        g = tg.gated_delta_rule_backward(dy, *args, saved, **more)
        t = tg.gated_delta_rule_step(*tok, cache, dt_bias=more["dt_bias"])
        return [y, s, *[x for x in g], t]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    pool = torch.cuda.graph_pool_handle()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = work()
        graphs.append((g, out))
    for k in range(4):
        with torch.no_grad():
            args[2].copy_(torch.randn_like(args[2]))
        start = torch.randn_like(cache)
        cache.copy_(start)
        want = [t.clone() for t in work()]
        kept = cache.clone()
        cache.copy_(start)
        g, out = graphs[k % 2]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(cache, kept), k


def test_on_another_stream():
    c = Case(([90], False, 1, 1, 64, 64, "f16", False, False, 0))
    want = tg.gated_delta_rule(*c.args(), **c.more())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tg.gated_delta_rule(*c.args(), stream=s, **c.more())
    s.synchronize()
    assert torch.equal(got, want)


def test_broadcast_rows():
    """One row for all tokens (stride 0), and gradients where rows are so."""
    c = Case(([40, 40], False, 1, 2, 24, 16, "f32", False, False, 0))
    one = lambda t: t[:, :1].expand_as(t)  # noqa: E731
    args = [t if t.dim() == 1 else one(t) for t in c.args()]
    full = [t if t.dim() == 1 else t.contiguous() for t in args]
    ya, ka = tg.gated_delta_rule_train(*args, dt_bias=up(c.dt_bias))
    yb, kb = tg.gated_delta_rule_train(*full, dt_bias=up(c.dt_bias))
    dy = one(c.dev(c.dy))
    assert torch.equal(ya, yb)
    for a, b in zip(tg.gated_delta_rule_backward(dy, *args, ka, dt_bias=up(c.dt_bias)),
                    tg.gated_delta_rule_backward(dy.contiguous(), *full, kb, dt_bias=up(c.dt_bias))):
        assert a is b or torch.equal(a, b)


def test_many_sequences():
    """More workgroups than the chip holds at once, against batches of a few."""
    S, L = 700, 37
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
    q, k, v, dt, beta, A = r(S, L, 1, 32), r(S, L, 1, 32), r(S, L, 2, 16), r(S, L, 2), r(S, L, 2), -torch.ones(2).cuda()
    y, state = tg.gated_delta_rule(q, k, v, dt, A, beta, return_state=True)
    for lo in (0, 300, S - 5):
        cut = [t[lo:lo + 5] for t in (q, k, v, dt)]
        ys, ss = tg.gated_delta_rule(*cut, A, beta[lo:lo + 5], return_state=True)
        assert torch.equal(y[lo:lo + 5], ys) and torch.equal(state[lo:lo + 5], ss)


def test_no_tokens():
    """Dense batches of no token, and no sequence to step: states pass through."""
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=F16)  # noqa: E731
    A, init = torch.ones(2, device="cuda"), torch.randn(3, 2, 8, 4, device="cuda")
    args = (z(3, 0, 1, 8), z(3, 0, 1, 8), z(3, 0, 2, 4), z(3, 0, 2), A, z(3, 0, 2))
    y, state = tg.gated_delta_rule(*args, initial_state=init, return_state=True)
    assert y.shape == (3, 0, 2, 4) and torch.equal(state, init)
    y, saved = tg.gated_delta_rule_train(*args, initial_state=init)
    d = tg.gated_delta_rule_backward(y, *args, saved, initial_state=init, dstate=init * 2)
    assert torch.equal(d.dinitial_state, init * 2) and not d.dA.any()
    step = tg.gated_delta_rule_step(*[t if t.dim() == 1 else t[0] for t in args], init.clone())
    assert step.shape == (0, 2, 4)


def test_state_gradient_without_an_initial_state():
    c = Case(([70, 33], True, 1, 2, 24, 16, "f32", True, False, 0))
    c.initial = None
    x, bias, _, y, state, _, kap, chunks = c.want(True)
    want = torch.autograd.grad((y * c.dy.double()).sum() + (state * c.dstate.double()).sum(), x[2])
    _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **c.more())
    D.near("dv", got.dv, want[0], D.allowed(F32, kap, chunks, gradient=True), F32)


def test_two_streams_at_once():
    """Two calls in flight share nothing."""
    a, b = Case(([500], False, 2, 4, 64, 64, "bf16", False, False, 0)), Case(([400], False, 1, 2, 96, 40, "f16", False, False, 0), 1)
    sets = [(c.args(), c.more(), c.dev(c.dy)) for c in (a, b)]

    def work(k):
        args, more, dy = sets[k]
        y, saved = tg.gated_delta_rule_train(*args, **more)
        return [y] + [t for t in tg.gated_delta_rule_backward(dy, *args, saved, **more) if t is not None]
    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = work(k)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for k in range(2) for p, q in zip(got[k], want[k]))
