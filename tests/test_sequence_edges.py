"""The sequence operators' edges on the host: sizes that no launch holds are
refused before one. No call here reaches the GPU."""
from __future__ import annotations

import ctypes

import pytest

from conv2d_batchnorm_silu_amd import sequence as S
from test_sequence_abi import F16, F32, P, UNSUP, _conv, _rows, _scan


@pytest.fixture(scope="module")
def lib():
    return S._lib()


@pytest.mark.parametrize("D,dtype,n", [(8, F16, 1 << 28), (130, F32, 1 << 26), (516, F32, 1 << 24),
                                       (513, F16, 1 << 24), (129, F16, 1 << 24)])
def test_conv_more_than_a_launch_holds(lib, D, dtype, n):
    """n rows, one to a sequence: with their states to write, or as single
    tokens, 2^32 threads or more along one axis."""
    rows = _rows(seq=D, row=D)
    a = _conv(seqs=n, rows=n, D=D, dtype=dtype, x=rows, y=rows, final=P)
    assert lib.tg_causal_conv(ctypes.byref(a), 0) == UNSUP
    assert lib.tg_causal_conv_backward(ctypes.byref(a), rows, rows, P, P, 0, P, P, 1 << 62, 0) == UNSUP
    assert lib.tg_causal_conv_step(P, D, P, n, 0, P, 0, n, D, 4, dtype, 0, P, 0) == UNSUP


@pytest.mark.parametrize("D,n", [(8, 1 << 24), (48, 1 << 24), (128, 1 << 23), (1000, 1 << 20)])
def test_scan_step_more_than_a_launch_holds(lib, D, n):
    rows, bc = _rows(seq=D, row=D), _rows(seq=16, row=16)
    a = _scan(seqs=n, rows=n, D=D, x=rows, dt=rows, z=rows, y=rows, B=bc, C=bc)
    assert lib.tg_selective_scan_step(ctypes.byref(a), P, n, 0, 0) == UNSUP
