"""The gated delta rule in segments against the 64-bit reference: the batches that
test_delta_segments.py shows to be cut, forward and backward."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import delta_ref as D
from test_delta_gpu import Case
from test_delta_gpu import test_backward as backward
from test_delta_gpu import test_forward as forward
from test_delta_precision_gpu import off
from test_delta_segments import CUT, is_cut

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", CUT, ids=str)
def test_cut_forward(case):
    assert is_cut(case)
    forward(case)


@pytest.mark.parametrize("case", CUT, ids=str)
def test_cut_backward(case):
    assert is_cut(case)
    backward(case)


@pytest.mark.parametrize("case", CUT, ids=str)
def test_cut_states_are_held_to_fp32(case):
    """As in test_delta_precision_gpu.py: independent roundings of all chunks by their
    squares, of three walks (to the segments' maps, between them, and from them)."""
    c = Case(case)
    _, _, _, y, state, _, kap, chunks = c.want()
    got, s = tg.gated_delta_rule(*c.args(), return_state=True, **c.more())
    allowed = 2 * (3 * chunks * D.STEPS) ** 0.5 * kap * D.E
    assert off(s, state) <= allowed, "%.3g, allowed %.3g" % (off(s, state), allowed)
    if c.dtype is torch.float32:
        assert off(got.reshape(y.shape), y) <= allowed, "%.3g, allowed %.3g" % (off(got.reshape(y.shape), y), allowed)
