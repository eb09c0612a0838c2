"""Which batches the gated delta rule walks in segments, seen from its scratch on the host
(no call here reaches the GPU): a batch that is not cut takes as much for each chunk,
whatever sequences they belong to."""
from __future__ import annotations

import ctypes

import pytest

from conv2d_batchnorm_silu_amd import sequence as S
from test_delta_abi import _delta
from test_sequence_abi import BF16, F16, F32, OK, P

TYPES = {"f16": F16, "bf16": BF16, "f32": F32}

# lengths, packed, key heads, value heads, K, V, type, state, plain gates and keys, extra
# row width: every type, dense and packed, several sequences, none, one token, lengths
# that are no multiple of a segment or a chunk.
CUT = [
    ([3001], False, 1, 2, 64, 40, "bf16", True, False, 0), ([2500, 2500], False, 1, 1, 64, 48, "bf16", True, False, 0),
    ([2100, 30, 0, 2170], True, 1, 2, 64, 40, "bf16", True, False, 3), ([0, 2600, 1], True, 2, 2, 128, 32, "bf16", False, False, 0),
    ([1900], False, 1, 1, 200, 40, "bf16", True, True, 0), ([1300, 1300], False, 1, 2, 48, 24, "f32", True, False, 0),
    ([0, 1201, 0, 900, 0], True, 1, 1, 32, 16, "f32", True, False, 0), ([1205, 1205, 1205], False, 1, 1, 64, 16, "f16", True, False, 0),
    ([700, 0, 1500], True, 1, 2, 100, 33, "f16", True, False, 0), ([1100], False, 1, 1, 130, 20, "f32", False, False, 0),
]


def work(seqs, rows, offsets, HK, HV, K, V, dt):
    a = _delta(seqs=seqs, rows=rows, offsets=offsets, HK=HK, HV=HV, K=K, V=V, dtype=TYPES[dt])
    size = ctypes.c_size_t()
    assert S._lib().tg_gated_delta_rule_sizes(ctypes.byref(a), ctypes.byref(size), None, None) == OK
    return size.value


def is_cut(case):
    lengths, packed, HK, HV, K, V, dt = case[:7]
    C = 64 if dt == "bf16" and K <= 128 else 32
    n, rows = len(lengths), sum(lengths)
    chunks = rows // C + n if packed else n * -(-lengths[0] // C)
    return work(n, rows, P if packed else 0, HK, HV, K, V, dt) > chunks * work(1, C, 0, HK, HV, K, V, dt)


@pytest.mark.parametrize("case", CUT, ids=str)
def test_cut(case):
    assert is_cut(case)


def test_short_and_full_batches_are_whole():
    assert not is_cut(([500], False, 1, 1, 64, 64, "bf16")) and not is_cut(([4096] * 64, False, 16, 16, 128, 128, "bf16"))
