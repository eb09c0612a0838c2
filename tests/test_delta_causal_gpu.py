"""What a NaN or an infinity reaches in the gated delta rule: its own token and later
ones of its head, of v its column alone; not the tokens before it, whatever they share."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
from gpu_cases import note
from test_delta_gpu import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# Chunks of 64 and 32 tokens, all widths, tails, few long sequences in segments.
CASES = [([150], False, 2, 4, 64, 40, "bf16", True, False, 0), ([64, 70], True, 1, 2, 128, 96, "bf16", True, False, 0),
         ([100], False, 1, 2, 200, 33, "bf16", False, True, 0), ([90], False, 2, 2, 60, 32, "f16", True, False, 0),
         ([80], False, 1, 1, 256, 48, "f16", True, False, 0), ([90], False, 1, 2, 32, 16, "f32", True, True, 3),
         ([70], False, 1, 1, 130, 40, "f32", True, False, 0), ([40, 0, 33], True, 1, 2, 256, 16, "f32", True, False, 0),
         ([2900], False, 1, 1, 32, 16, "bf16", True, False, 0), ([1500], False, 1, 2, 40, 20, "f32", True, False, 0)]


def run(c, train):
    more = dict(c.more(), return_state=True)
    if train:
        return tg.gated_delta_rule_train(*c.args(), **more)[:2]
    return tg.gated_delta_rule(*c.args(), **more)


def rows(c, y):
    return y.reshape(c.T, c.HV, -1)


def same(a, b):
    return torch.equal(a, b)


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_tokens_before_a_bad_one(case, train):
    note("delta bad values %s %s" % (case, train))
    c = Case(case)
    y0, s0 = run(c, train)
    y0 = rows(c, y0)
    HK, HV = c.k.shape[1], c.HV
    rep, last, V = HV // HK, len(c.lengths) - 1, c.v.shape[-1]
    lo, hi = c.bounds[last], c.bounds[last + 1]
    n = hi - lo
    gates = ("dt", "beta")
    for at in sorted({lo, lo + 1, lo + min(17, n - 1), lo + min(31, n - 1), lo + n // 2, hi - 1}):
        for name in ("v", "k", "q") + gates:
            for bad in (NAN, INF) if name not in gates else (NAN,):
                held = getattr(c, name)
                t = held.clone()
                h = t.shape[1] - 1
                if name in gates:
                    t[at, h] = bad
                else:
                    t[at, h, t.shape[2] // 2] = bad
                setattr(c, name, t)
                y, s = run(c, train)
                setattr(c, name, held)
                y = rows(c, y)
                what = (name, bad, at)
                assert same(y[:at], y0[:at]), what
                heads = slice(0, HV - (rep if name in ("k", "q") else 1))  # of others
                assert same(y[:, heads], y0[:, heads]) and same(s[:, heads], s0[:, heads]), what
                assert same(s[:last], s0[:last]), what
                if name == "q":
                    assert same(y[at + 1:], y0[at + 1:]) and same(s, s0), what
                    assert not torch.isfinite(y[at, h * rep:]).any(), what
                elif name == "v":
                    keep = [v for v in range(V) if v != V // 2]
                    assert same(y[..., keep], y0[..., keep]) and same(s[..., keep], s0[..., keep]), what
                    assert not torch.isfinite(y[at:, h, V // 2]).any(), what
                else:
                    own = slice(h * rep, HV) if name == "k" else slice(h, h + 1)
                    assert not torch.isfinite(y[at:, own]).any() and not torch.isfinite(s[last, own]).all(), what


@pytest.mark.parametrize("case", CASES[:8], ids=str)
def test_rows_of_nothing_behind_a_sequence(case):
    """A padded batch whose rows past the real tokens hold NaN in every tensor."""
    c = Case(case)
    y0 = rows(c, run(c, False)[0])
    last = len(c.lengths) - 1
    at = c.bounds[last] + c.lengths[last] // 2 + 1
    for name in ("q", "k", "v", "dt", "beta"):
        t = getattr(c, name).clone()
        t[at:c.bounds[last + 1]] = NAN
        setattr(c, name, t)
    y = rows(c, run(c, False)[0])
    assert same(y[:at], y0[:at])


def test_an_initial_state_that_is_none():
    """A column of NaN stays in its column."""
    c = Case(CASES[0])
    y0, s0 = run(c, False)
    c.initial = c.initial.clone()
    c.initial[0, 1, 5, 7] = NAN
    y, s = run(c, False)
    keep = [v for v in range(40) if v != 7]
    assert same(y[..., keep], y0[..., keep]) and same(s[..., keep], s0[..., keep])
    assert bool(torch.isnan(y[0, :, 1, 7]).all())
