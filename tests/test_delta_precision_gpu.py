"""What the gated delta rule's outputs may be off beside the rounding of their type,
held more tightly than the worst cases of delta_ref.py: by root sums of squares.

A 2-norm over thousands of elements adds independent roundings up by their squares.
With delta_ref's counts (fewer than STEPS roundings of u = 2^-24 each on the way from
one chunk's state to the next, amplified by KAPPA) the states after n chunks are off
by less than sqrt(n STEPS) KAPPA u of their norm; twice that is allowed."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import delta_ref as D
from gpu_cases import note
from test_delta_gpu import Case, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# A chunk or three, all types and widths of both chunk lengths, states and gates.
SHORT = [
    ([64], False, 2, 2, 64, 64, "bf16", True, False, 0), ([64, 64], False, 1, 2, 128, 96, "bf16", True, False, 0),
    ([96], False, 1, 2, 96, 81, "f16", True, False, 0), ([70, 0, 33], True, 1, 2, 64, 48, "f16", True, False, 3),
    ([90], False, 1, 1, 200, 64, "bf16", True, False, 0), ([64], False, 1, 1, 256, 40, "f16", True, False, 0),
    ([60], False, 2, 2, 64, 64, "f32", True, False, 0), ([80], False, 1, 2, 256, 33, "f32", True, False, 0),
]


def off(got, want):
    d = got.detach().double().cpu() - want
    return float(d.norm() / want.norm())


@pytest.mark.parametrize("case", SHORT, ids=str)
def test_states_are_held_to_fp32(case):
    note("delta states %s" % (case,))
    c = Case(case)
    _, _, _, _, state, _, kap, chunks = c.want()
    _, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
    allowed = 2 * (chunks * D.STEPS) ** 0.5 * kap * D.E
    assert off(s, state) <= allowed, "%.3g, allowed %.3g" % (off(s, state), allowed)


@pytest.mark.parametrize("case", SHORT + [([3300], True, 1, 2, 64, 40, "bf16", True, False, 0)], ids=str)
def test_prompts_and_training_are_the_same(case):
    """What is kept for the gradients does not change what comes out."""
    c = Case(case)
    y, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
    y2, s2, _ = tg.gated_delta_rule_train(*c.args(), return_state=True, **c.more())
    assert torch.equal(y, y2) and torch.equal(s, s2)


@pytest.mark.parametrize("case", [c for c in SHORT if c[6] != "f32"], ids=str)
def test_gradients_of_q_and_k_round_once(case):
    """An error of e, relative to the value, moves it past the middle between two
    numbers of its type in a share 2 e / step of all elements, with step at least eps/2
    of the value. What leads to dq and dk is off by three operands of 2^-17 (two parts and
    the product of two second ones) and by fp32's roundings, of what an element is a
    difference of; four standard deviations of the count are added."""
    note("delta dq, dk %s" % (case,))
    c = Case(case)
    x, bias, initial, y, state, g, kap, chunks = c.want(True)
    total = (y * c.dy.double()).sum() + (state * c.dstate.double()).sum()
    dq, dk, uq, uk = torch.autograd.grad(total, [x[0], x[1], g[1], g[2]])
    _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **c.more())
    e = 3 * 2.0 ** -17 + 2 * (chunks * D.STEPS) ** 0.5 * kap * kap * D.E
    for name, want, at, unit in (("dq", dq, 0, uq), ("dk", dk, 1, uk)):
        size = torch.maximum(want.abs(), D.unit_size(x[at].detach(), unit))
        rms = size.norm() / size.numel() ** 0.5
        half = torch.finfo(c.dtype).eps / 2
        share = (2 * e * torch.maximum(size, rms) / (want.abs() * half)).clamp(max=1)
        n = int((getattr(got, name).cpu().reshape(want.shape) != want.to(c.dtype)).sum())
        most = float(share.sum()) + 4 * float((share * (1 - share)).sum()) ** 0.5 + 1
        assert n <= most, "%s: %d of %d not the rounded value, allowed %.0f" % (name, n, want.numel(), most)


@pytest.mark.parametrize("case", [c for c in SHORT if c[6] == "f32"], ids=str)
def test_gradients_of_fp32_by_their_squares(case):
    """Through both walks, twice the roundings of one and KAPPA for each; of what an
    element is a difference of, for q and k."""
    note("delta fp32 gradients %s" % (case,))
    c = Case(case)
    x, bias, initial, y, state, g, kap, chunks = c.want(True)
    total = (y * c.dy.double()).sum() + (state * c.dstate.double()).sum()
    want = torch.autograd.grad(total, x + [initial, g[1], g[2]])
    _, saved = tg.gated_delta_rule_train(*c.args(), **c.more())
    got = tg.gated_delta_rule_backward(c.dev(c.dy), *c.args(), saved, dstate=up(c.dstate), **c.more())
    allowed = 2 * (2 * chunks * D.STEPS) ** 0.5 * kap * kap * D.E
    for name, w, size in (("dq", want[0], D.unit_size(x[0].detach(), want[7])), ("dk", want[1], D.unit_size(x[1].detach(), want[8])),
                          ("dv", want[2], want[2]), ("ddt", want[3], want[3]), ("dbeta", want[5], want[5]),
                          ("dinitial_state", want[6], want[6])):
        d = float((getattr(got, name).double().cpu().reshape(w.shape) - w).norm() / torch.maximum(size.abs(), w.abs()).norm())
        assert d <= allowed, "%s: %.3g, allowed %.3g" % (name, d, allowed)
